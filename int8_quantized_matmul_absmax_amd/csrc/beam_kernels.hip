// A beam search's choice of its next beams: the best of beams x vocabulary.
//
// A candidate's value is s_i + x_iv - log sum_u exp(x_iu), with s the beam's
// score and x its logits. Within a beam the order is the logits' own, so a first
// kernel reads each row once, in pieces, and leaves of each its maximum, its sum
// of exponentials and its best `count` logits; a second one makes the rows' sums
// whole and takes the best of the pieces' best.
//
// Values of different beams are compared in 64 bits: rounded to 32 bits, scores
// of some tens would make ties of candidates that are apart. Sums of
// exponentials are 32-bit within a lane and 64-bit from there on.

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"

namespace i8mm {

namespace {

constexpr int kWaves = kBlockThreads / kWave;
constexpr int kVectors = 4;   // 16-byte loads a lane takes at once
// log2(e) to 24 bits, and what it is off by relative to itself.
constexpr float kLog2E = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417;
constexpr float kLeastWord = -3.402823466e38f;   // of fp32
constexpr double kOff = (double)kLog2E * kLn2 - 1.0;

// 16 bytes of a row, which begins at any element.
struct __attribute__((packed, aligned(2))) Loose16 {
  v4i32 x;
};

// Whole-wave shift by one lane: lane l gets lane l - 1's (DPP wave_shr:1).
__device__ __forceinline__ uint32_t from_lane_below(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x138, 0xf, 0xf, false);
}

// What a piece leaves: its base and its sum (the logits' exponentials add up to sum
// times 2^base for fp16, e^base for fp32), then `count` values and as many indices, best first.
struct Pieces {
  float2* sum;      // [rows][pieces]
  float* value;     // [rows][pieces][count]
  uint32_t* index;
};
__host__ __device__ __forceinline__ Pieces pieces_of(void* ws, int64_t rows, int pieces, int count) {
  Pieces p;
  p.sum = static_cast<float2*>(ws);
  p.value = reinterpret_cast<float*>(p.sum + rows * pieces);
  p.index = reinterpret_cast<uint32_t*>(p.value + rows * pieces * count);
  return p;
}

// The order of floats as integers, zeros of both signs equal.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A word's key: its value, then its index, lower ones first. Keys are unique; kNoKey is
// not less than that of a word of -infinity.
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  return (uint64_t)order_of(x) << 32 | (uint32_t)~i;
}
constexpr uint64_t kNoKey = 0x007fffffffffffffull;
__device__ __forceinline__ int lanes_before(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// A wave's words that may be among the piece's best, in any order, in LDS. When there is
// no room for more they become their `count` best, and what a word has to beat the least
// of those.
constexpr int kHold = 256;
struct Hold {
  uint64_t* key;
  int n = 0;
  uint64_t least = kNoKey;
  __device__ __forceinline__ void shrink(int count, int lane) {
    uint64_t k[kHold / kWave];
#pragma unroll
    for (int j = 0; j < kHold / kWave; ++j)
      k[j] = j * kWave + lane < n ? key[j * kWave + lane] : 0;
    // the key of place `count`, bit by bit: of the values, then, of more words of the last
    // value than there are places, of the indices (below 2^17: a piece's)
    auto reach = [&](uint64_t least) __attribute__((always_inline)) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < kHold / kWave; ++j) n += __popcll(__ballot(k[j] >= least));
      return n;
    };
    uint64_t t = 0;
#pragma unroll 1
    for (uint64_t bit = 1ull << 63; bit > 0xffffffffull; bit >>= 1)
      if (reach(t | bit) >= count) t |= bit;
    if (reach(t) > count) {
      t |= 0xfffe0000u;
#pragma unroll 1
      for (uint64_t bit = 0x10000; bit; bit >>= 1)
        if (reach(t | bit) >= count) t |= bit;
    }
    least = t;
    n = 0;
#pragma unroll
    for (int j = 0; j < kHold / kWave; ++j) {
      const uint64_t those = __ballot(k[j] >= t);
      if (k[j] >= t) key[n + lanes_before(those)] = k[j];
      n += __popcll(those);
    }
  }
  // (the wave together; `some`: of lanes that have one)
  __device__ __forceinline__ void add(bool some, uint64_t k, int count, int lane) {
    uint64_t those = __ballot(some && k > least);
    if (n + __popcll(those) > kHold) {
      shrink(count, lane);
      those = __ballot(some && k > least);
    }
    if (some && k > least) key[n + lanes_before(those)] = k;
    n += __popcll(those);
  }
};

// 2^d, or e^d of a base in the logits' own units.
__device__ __forceinline__ float power_of(float d, bool natural) {
  return __builtin_amdgcn_exp2f(natural ? d * kLog2E : d);
}

// A value that `count` of kN x of each lane reach (-infinity where fewer are more than
// that), within 2^-7 of the largest such: the order of floats, its upper 16 bits searched
// bit by bit.
template <int kN>
__device__ __forceinline__ float reached_by(const float (&x)[kN], int count) {
  uint32_t key[kN];
#pragma unroll
  for (int w = 0; w < kN; ++w) key[w] = order_of(x[w]) >> 16;
  uint32_t t = 0;
#pragma unroll
  for (uint32_t bit = 0x8000u; bit; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kN; ++w) n += __popcll(__ballot(key[w] >= (t | bit)));
    if (n >= count) t |= bit;
  }
  return t <= 0x007fu ? -INFINITY : of_order(t << 16);
}

// A lane's 16 bytes of a row, and their greatest element.
template <bool kHalf>
struct Words {
  static constexpr int kV = kHalf ? 8 : 4;
  v4i32 raw;
  __device__ __forceinline__ float at(int e) const {
    if constexpr (kHalf)
      return h2f(((uint32_t)raw[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    else
      return __builtin_bit_cast(float, (uint32_t)raw[e]);
  }
  // (a lane's own e)
  __device__ __forceinline__ float pick(int e) const {
    const int w = kHalf ? e >> 1 : e;
    const uint32_t lo = (uint32_t)(w & 1 ? raw[1] : raw[0]), hi = (uint32_t)(w & 1 ? raw[3] : raw[2]);
    const uint32_t x = w & 2 ? hi : lo;
    if constexpr (kHalf)
      return h2f((x >> (16 * (e & 1))) & 0xffffu);
    else
      return __builtin_bit_cast(float, x);
  }
  __device__ __forceinline__ float most() const {
    if constexpr (kHalf) {
      v2f16 m = __builtin_bit_cast(v2f16, (uint32_t)raw[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(v2f16, (uint32_t)raw[e]));
      return fmaxf((float)m[0], (float)m[1]);
    } else {
      return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3)));
    }
  }
  // 2^(x L - b) of element e, for fp32 2^((x - b) L)
  __device__ __forceinline__ float power(int e, float b) const {
    float y;
    if constexpr (kHalf) {
      if (e & 1)
        asm("v_fma_mix_f32 %0, %1, %2, -%3 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
            : "=v"(y) : "v"(raw[e >> 1]), "s"(kLog2E), "v"(b));
      else
        asm("v_fma_mix_f32 %0, %1, %2, -%3 op_sel:[0,0,0] op_sel_hi:[1,0,0]"
            : "=v"(y) : "v"(raw[e >> 1]), "s"(kLog2E), "v"(b));
    } else {
      y = (at(e) - b) * kLog2E;
    }
    return __builtin_amdgcn_exp2f(y);
  }
  // Words from i on. A row's last ones are taken by a lane that begins before them:
  // `drop` of its words are another's, and -infinity here.
  __device__ __forceinline__ void load(const int8_t* row, int i) {
    raw = reinterpret_cast<const Loose16*>(row + (int64_t)i * (16 / kV))->x;
  }
  __device__ __forceinline__ void drop(int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kHalf) {
        const uint32_t w = (uint32_t)raw[e];
        const uint32_t lo = 2 * e < n ? 0xfc00u : w & 0xffffu;
        raw[e] = (int)((2 * e + 1 < n ? 0xfc000000u : w & 0xffff0000u) | lo);
      } else {
        raw[e] = e < n ? (int)0xff800000u : raw[e];
      }
    }
  }
  // Of a row of fewer than kV words, the first n.
  __device__ __forceinline__ void load_few(const int8_t* row, int n) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      if constexpr (kHalf) {
        const uint32_t h = e < n ? reinterpret_cast<const uint16_t*>(row)[e] : 0xfc00u;
        raw[e >> 1] = (int)(e & 1 ? (uint32_t)raw[e >> 1] | h << 16 : h);
      } else {
        raw[e] = e < n ? reinterpret_cast<const int32_t*>(row)[e] : (int)0xff800000u;
      }
    }
  }
};

// One block a piece. A wave takes 4 KB at a time, the next in flight meanwhile.
//
// Exponentials are 2^(x L - b) with L = log2(e) to 24 bits and any b near the maximum:
// one fma that takes x in its 16 bits, whose rounding matters little where the result
// is large, and b is known exactly. L is log2(e) (1 + kOff), so what is summed are
// exponentials of x (1 + kOff), and their logarithm is off by kOff times the mean of
// x under the softmax; the join takes kOff times the maximum off instead. Of fp32
// logits, whose product with L may overflow, (x - b) L with b the maximum itself.
//
// The best words are held unsorted until the end. What keeps them few is a floor, a value
// that `count` of the block's words reach: the block's first 16 KB set one, what `count`
// of its lanes' maxima reach; later it is the least of what a wave's share of `count` of
// its lanes' maxima reach, over the waves. (Sorted over a wave's lanes as they come,
// with an insertion of about 100 instructions for each: 264 rows of 139286 fp16 words
// with 24 places 36 us in place of 30, 80 of 50257 fp32 words with 10 12.2 and 10.6.)
//
// 512 rows of 131072 fp16 words: 31 us, 4.3 TB/s, of which the first and the last words
// and the sorting take 6; 4 rows of 32000 words 6.7 us, a chain of waits.
template <bool kHalf, bool kFew>
__global__ __launch_bounds__(kBlockThreads) void k_beam_rows(BeamArgs a, int pieces, int piece) {
  typedef Words<kHalf> W;
  constexpr int kV = W::kV, kStep = kVectors * kWave * kV;
  __shared__ float s_x[kBlockThreads], s_b[kWaves], s_l[kWaves], s_share[kWaves];
  __shared__ uint64_t s_key[kWaves][kHold];
  __shared__ int s_n[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = blockIdx.x / pieces, at_piece = blockIdx.x % pieces;
  if (a.live && a.live[row] == 0) return;   // the join reads nothing of it
  const int64_t begin = (int64_t)at_piece * piece;
  const int n = (int)min((int64_t)piece, a.vocab - begin);
  const int8_t* const words =
      static_cast<const int8_t*>(a.logits) + (row * a.row_stride + begin) * (kHalf ? 2 : 4);
  if (threadIdx.x < kWaves) s_share[threadIdx.x] = -INFINITY;

  Hold hold;
  hold.key = s_key[wave];
  float b = 0.f, l = 0.f;   // of the lane: l 2^b
  bool any = false;
  float floor = -INFINITY, top_so_far = -INFINITY;
  W x[kVectors], ahead[kVectors];
  // (before the piece's first word for a short piece, never before the row's)
  auto first = [&](int at, int u) __attribute__((always_inline)) {
    return min(at + (u * kWave + lane) * kV, n - kV);
  };
  auto load = [&](W (&to)[kVectors], int at) __attribute__((always_inline)) {
    if constexpr (kFew) return;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) to[u].load(words, first(at, u));
  };
  int at = wave * kStep;
  load(x, at);
  for (bool start = true; start || at < n; start = false, at += kWaves * kStep) {
    load(ahead, at + kWaves * kStep);   // (past the end, the last words again)
    if constexpr (kFew) {
#pragma unroll
      for (int u = 0; u < kVectors; ++u)
        x[u].load_few(words, wave == 0 && lane == 0 && u == 0 ? n : 0);
    } else if (at + kStep > n) {
#pragma unroll
      for (int u = 0; u < kVectors; ++u) x[u].drop(at + (u * kWave + lane) * kV - first(at, u));
    }
    float top[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) top[u] = x[u].most();
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    top_so_far = fmaxf(top_so_far, most);
    if (start) {
      s_x[threadIdx.x] = most;
      lds_only_barrier();
      float all[kWaves];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) all[w] = s_x[w * kWave + lane];
      floor = fmaxf(reached_by(all, a.count), kLeastWord);
    } else {
      // (what a wave reads may be older than what others have written since: they only
      // rise. Not volatile: that is a load which waits for the logits in flight, too.)
      float least = INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        least = fminf(least, __hip_atomic_load(&s_share[w], __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_WORKGROUP));
      floor = fmaxf(floor, least);
    }

    // A NaN or +infinity makes the sum NaN, and the row one without candidates.
    const float next = kHalf ? most * kLog2E : most;
    if (most > -INFINITY && (!any || next > b)) {
      l *= any ? power_of(b - next, !kHalf) : 0.f;
      b = next;
      any = true;
    }
    float sum[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      sum[u] = 0.f;
#pragma unroll
      for (int e = 0; e < kV; ++e)
        sum[u] += x[u].power(e, b);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);

    const auto index = [&](int u) __attribute__((always_inline)) {
      return kFew ? 0 : first(at, u);
    };
    if (__any(most >= floor)) {
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        if (!__any(top[u] >= floor)) continue;
        uint32_t those = 0;   // of the lane's words, a bit each
#pragma unroll
        for (int e = 0; e < kV; ++e) those |= x[u].at(e) >= floor ? 1u << e : 0u;
        while (__any(those != 0)) {
          const int e = those ? __builtin_ctz(those) : 0;
          hold.add(those != 0, key_of(x[u].pick(e), index(u) + e), a.count, lane);
          those &= those - 1;   // (of none, none)
        }
      }
      const float own[1] = {top_so_far};
      const float reached = reached_by(own, (a.count + kWaves - 1) / kWaves);
      if (lane == 0)
        __hip_atomic_store(&s_share[wave], reached, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u] = ahead[u];
  }

  // the wave's sum, then the block's
  const float mine = any ? b : -INFINITY;
  float top = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  l *= any ? power_of(mine - top, !kHalf) : 1.f;   // (nothing: 0, or a NaN)
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) l += __shfl_xor(l, d, kWave);
  if (lane == 0) {
    s_b[wave] = top;
    s_l[wave] = l;
  }
  if (lane == 0) s_n[wave] = hold.n;
  __syncthreads();
  if (s_n[0] + s_n[1] + s_n[2] + s_n[3] > kBlockThreads) {
    // (count of each wave's are at most a block's threads)
    __syncthreads();
    if (hold.n > a.count) hold.shrink(a.count, lane);
    if (lane == 0) s_n[wave] = hold.n;
    __syncthreads();
  }
  const Pieces out = pieces_of(a.ws, (int64_t)a.batch * a.beams, pieces, a.count);
  const int64_t part = (int64_t)row * pieces + at_piece;
  // An entry's place is the number of entries before it; lanes share an entry.
  int n_of[kWaves], entries = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    n_of[w] = __builtin_amdgcn_readfirstlane(s_n[w]);
    entries += n_of[w];
  }
  int lanes = 1;
  while (2 * lanes * entries <= kBlockThreads && lanes < kWave) lanes *= 2;
  int of_wave = 0, entry = threadIdx.x / lanes;
  const bool some = entry < entries;
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
    if (of_wave == w && entry >= n_of[w]) {
      entry -= n_of[w];
      ++of_wave;
    }
  const uint64_t key = some ? s_key[of_wave][entry] : 0;
  int place = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    for (int o = threadIdx.x % lanes; o < n_of[w]; o += lanes) place += s_key[w][o] > key;
  for (int d = 1; d < lanes; d <<= 1) place += __shfl_xor(place, d, kWave);
  if (some && threadIdx.x % lanes == 0 && place < a.count) {
    out.value[part * a.count + place] = of_order((uint32_t)(key >> 32));
    out.index[part * a.count + place] = ~(uint32_t)key + (uint32_t)begin;
  }
  for (int j = entries + threadIdx.x; j < a.count; j += kBlockThreads) {
    out.value[part * a.count + j] = -INFINITY;
    out.index[part * a.count + j] = 0;
  }
  if (threadIdx.x == 0) {
    float t = s_b[0], sum = 0.f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t = fmaxf(t, s_b[w]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum += s_b[w] > -INFINITY ? s_l[w] * power_of(s_b[w] - t, !kHalf) : s_l[w];
    out.sum[part] = float2{t, sum};
  }
}

// 64-bit words of a lane.
__device__ __forceinline__ uint64_t lane_word(uint64_t x, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ double lane_double(double x, int lane) {
  return __builtin_bit_cast(double, lane_word(__builtin_bit_cast(uint64_t, x), lane));
}
__device__ __forceinline__ uint64_t word_from_lane_below(uint64_t x) {
  return (uint64_t)from_lane_below((uint32_t)(x >> 32)) << 32 | from_lane_below((uint32_t)x);
}
// -infinity from a word that the compiler does not look into: where it keeps the
// constant in a pair of scalar registers, it sets them with one s_mov_b64, whose
// literal has 32 bits, and they hold 0 (hipcc of ROCm 7.2).
__device__ __forceinline__ double no_value() {
  uint32_t high = 0xfff00000u;
  asm volatile("" : "+s"(high));
  return __builtin_bit_cast(double, (uint64_t)high << 32);
}
// Whether candidate (v, at) comes before (w, bt); `at` counts beams x vocabulary.
__device__ __forceinline__ bool before(double v, int64_t at, double w, int64_t bt) {
  return v > w || (v == w && at < bt);
}

// The upper bits of a value's order, and the least value that has them.
constexpr int kHeadBits = 24;
__device__ __forceinline__ uint32_t head_of(double x) {
  const uint32_t b = (uint32_t)(__builtin_bit_cast(uint64_t, x) >> 32);
  return (b ^ ((uint32_t)((int)b >> 31) | 0x80000000u)) >> (32 - kHeadBits);
}
__device__ __forceinline__ double of_head(uint32_t k) {
  const uint32_t o = k << (32 - kHeadBits);
  const bool positive = o & 0x80000000u;
  const uint32_t high = positive ? o ^ 0x80000000u : ~o, low = positive ? 0u : 0xffffffffu;
  return __builtin_bit_cast(double, (uint64_t)high << 32 | low);
}

// One block a search.
//
// A beam's base, what its logits are added to: its score less the logarithm, of which
// the integer part and the 24-bit logarithm of the rest are put together in 64 bits.
// A candidate's place is the number of candidates before it, counted over all pairs of
// up to kJoinEntries; more of them first become the lists of the block's waves. Bound by
// waits: the sums 1.7 us, the lists' last places 1.1, the candidates 1.7, their places
// 0.7; 4 us with few, 7 with 350.
// (Fewer than kJoinFew are counted at once: 4 beams of 4 pieces' 4 10.5 us in all, with a
// bound for them first 11.8; 13 pieces' 16 17.9 and 17.2.)
constexpr int kJoinFew = 64;
constexpr int kJoinMany = 128;
constexpr int kJoinAhead = 4;   // candidates of a thread in flight
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave;
constexpr int kJoinEntries = kJoinWaves * I8MM_MAX_BEAM_COUNT;
__global__ __launch_bounds__(kJoinThreads) void k_beam_join(BeamArgs a, int pieces) {
  extern __shared__ double s_base[];   // [beams], then whether they have ended
  int* const s_ended = reinterpret_cast<int*>(s_base + a.beams);
  __shared__ double s_v[kJoinEntries];
  __shared__ int64_t s_at[kJoinEntries];
  __shared__ int s_count;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x;
  const Pieces in = pieces_of(a.ws, (int64_t)a.batch * a.beams, pieces, a.count);
  for (int i = wave; i < a.beams; i += kJoinWaves) {
    const int64_t row = (int64_t)b * a.beams + i;
    const float s = a.scores[row];
    const bool ended = a.live && a.live[row] == 0;
    double base = fabsf(s) < INFINITY ? (double)s : no_value();
    if (!ended) {
      float top = -INFINITY, sum = 0.f;
      for (int p = lane; p < pieces; p += kWave) {
        const float2 x = in.sum[row * pieces + p];
        const float next = fmaxf(top, x.x);
        sum = sum * (top > -INFINITY ? power_of(top - next, a.fp32) : 1.f) +
              x.y * (x.x > -INFINITY ? power_of(x.x - next, a.fp32) : 1.f);
        top = next;
      }
      float all = top;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) all = fmaxf(all, __shfl_xor(all, d, kWave));
      double total = (double)(sum * (top > -INFINITY ? power_of(top - all, a.fp32) : 1.f));
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) total += __shfl_xor(total, d, kWave);
      const int e = __builtin_amdgcn_frexp_exp(total);
      const float rest = __builtin_amdgcn_logf((float)__builtin_amdgcn_frexp_mant(total));
      base -= ((double)e + (double)rest) * kLn2;
      base -= a.fp32 ? (double)all : (double)all * (kLn2 - kLn2 * kOff);
      if (!(total > 0.0) || !(total < 1e300)) base = no_value();
    }
    if (lane == 0) {
      s_base[i] = base;
      s_ended[i] = ended;
    }
  }
  __syncthreads();

  const double none = no_value();
  // (no words: a beam that has ended still has its one candidate)
  const int per_beam = max(pieces * a.count, 1), all = a.beams * per_beam;
  const int64_t words = max(a.vocab, (int64_t)1);
  // (loaded whether it is one or not, so that several can be in flight)
  const int64_t first = (int64_t)b * all;
  auto candidate = [&](int e, double* v, int64_t* at) __attribute__((always_inline)) {
    const int c = min(e, all - 1), i = c / per_beam;
    const double base = s_base[i];
    const bool ended = s_ended[i];
    const float x = pieces > 0 ? in.value[first + c] : 0.f;
    const int word = pieces > 0 ? (int)in.index[first + c] : 0;
    const double own = c == i * per_beam ? base : none;
    const double sum = ended ? own : base + (double)x;
    const bool some = e < all && sum > none;   // (not of an empty place, or a row without candidates)
    *v = some ? sum : none;
    *at = some ? i * words + (ended ? max(a.eos, 0) : word) : 0;
  };
  // Of more than kJoinFew, only those are counted that reach the last place of the list
  // with the best one: that list alone has `count` of them. If they are still more than
  // kJoinMany, as of many lists that are alike, only those that reach what `count` of 64
  // groups' best reach (groups of a lane of each wave, another one in each: a list's best
  // stand in neighbouring lanes).
  double least = none;
  if (all > kJoinFew) {
    const int lists = pieces > 0 ? a.beams * pieces : 0;
    for (int e = threadIdx.x; e < lists; e += kJoinThreads) {
      double v;
      int64_t at;
      candidate(e * a.count + a.count - 1, &v, &at);
      least = v > least ? v : least;
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_xor(least, d, kWave);
      least = o > least ? o : least;
    }
    if (lane == 0) s_v[wave] = least;
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    least = s_v[0];
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) least = s_v[w] > least ? s_v[w] : least;
    __syncthreads();
    double mine = none;   // the best of the thread's
    auto sweep = [&](auto ahead) __attribute__((always_inline)) {
      constexpr int kN = decltype(ahead)::value;
      for (int e0 = 0; e0 < all; e0 += kN * kJoinThreads) {
        double v[kN];
        int64_t at[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u)
          candidate(e0 + u * kJoinThreads + threadIdx.x, &v[u], &at[u]);
#pragma unroll
        for (int u = 0; u < kN; ++u) {
          mine = v[u] > mine ? v[u] : mine;
          const bool some = v[u] > none && v[u] >= least;
          const uint64_t those = __ballot(some);
          if (!those) continue;
          int to = 0;
          if (lane == 0) to = atomicAdd(&s_count, __popcll(those));
          to = __builtin_amdgcn_readfirstlane(to) + lanes_before(those);
          if (some && to < kJoinEntries) {
            s_v[to] = v[u];
            s_at[to] = at[u];
          }
        }
      }
    };
    for (int round = 0;; ++round) {
      if (all <= kJoinThreads)
        sweep(std::integral_constant<int, 1>());
      else
        sweep(std::integral_constant<int, kJoinAhead>());
      __syncthreads();
      if (round == 1 || s_count <= kJoinMany) break;
      uint32_t* const s_head = reinterpret_cast<uint32_t*>(s_v);
      __syncthreads();
      s_head[threadIdx.x] = head_of(mine);
      if (threadIdx.x == 0) s_count = 0;
      __syncthreads();
      uint32_t head = 0, t = 0;
#pragma unroll
      for (int w = 0; w < kJoinWaves; ++w) head = max(head, s_head[w * kWave + ((lane + 5 * w) & 63)]);
#pragma unroll 1
      for (uint32_t bit = 1u << (kHeadBits - 1); bit; bit >>= 1)
        if (__popcll(__ballot(head >= (t | bit))) >= a.count) t |= bit;
      const double reached = of_head(t);   // (a NaN if fewer groups have one)
      least = reached > least ? reached : least;
      __syncthreads();
    }
  }
  int entries = all > kJoinFew ? s_count : all;
  if (all <= kJoinFew) {
    if ((int)threadIdx.x < all) candidate(threadIdx.x, &s_v[threadIdx.x], &s_at[threadIdx.x]);
  } else if (entries > kJoinEntries) {
    entries = kJoinWaves * a.count;
    double best = none, last = none;   // as in the rows' lists
    int64_t best_at = 0, last_at = 0;
    for (int e0 = wave * kWave; e0 < all; e0 += kJoinThreads) {
      double v;
      int64_t at;
      candidate(e0 + lane, &v, &at);
      uint64_t those = __ballot(v > none && before(v, at, last, last_at));
      while (those) {
        const int from = __builtin_ctzll(those);
        those &= those - 1;
        const double w = lane_double(v, from);
        const int64_t w_at = (int64_t)lane_word((uint64_t)at, from);
        if (!before(w, w_at, last, last_at)) continue;
        const int place = __popcll(__ballot(before(best, best_at, w, w_at)));
        const double up =
            __builtin_bit_cast(double, word_from_lane_below(__builtin_bit_cast(uint64_t, best)));
        const int64_t up_at = (int64_t)word_from_lane_below((uint64_t)best_at);
        best = lane < place ? best : lane == place ? w : up;
        best_at = lane < place ? best_at : lane == place ? w_at : up_at;
        last = lane_double(best, a.count - 1);
        last_at = (int64_t)lane_word((uint64_t)best_at, a.count - 1);
      }
    }
    if (lane < a.count) {
      s_v[wave * a.count + lane] = best;
      s_at[wave * a.count + lane] = best_at;
    }
  }
  __syncthreads();
  int lanes = 1;   // that share an entry
  while (2 * lanes * entries <= kJoinThreads && lanes < 16) lanes *= 2;
  const int entry = threadIdx.x / lanes;
  const double v = entry < entries ? s_v[entry] : none;
  const int64_t at = entry < entries ? s_at[entry] : 0;
  int place = 0;
#pragma unroll 4
  for (int o = threadIdx.x % lanes; o < entries; o += lanes) {
    const double ov = s_v[o];
    const int64_t o_at = s_at[o];
    // (empty places are equal)
    place += ov > v || (ov == v && (o_at < at || (o_at == at && o < entry)));
  }
  for (int d = 1; d < lanes; d <<= 1) place += __shfl_xor(place, d, kWave);
  if (threadIdx.x % lanes == 0 && place < a.count && (entry < entries)) {
    const bool found = v > none;
    const int64_t i = at / words;
    const int64_t to = (int64_t)b * a.count + place;
    const int64_t row = (int64_t)b * a.beams + i;
    // (where none is found, at is 0 and the row the search's first)
    const bool ended = a.live && a.live[row] == 0;
    const int token = ended ? a.eos : (int)(at - i * words);
    a.out_scores[to] = (float)v;
    a.out_tokens[to] = found ? token : -1;
    a.out_parents[to] = found ? (int)row : -1;
    a.out_live[to] = found && token != a.eos;
  }
  // places that no entry is left for
  for (int j = entries + threadIdx.x; j < a.count; j += kJoinThreads) {
    const int64_t to = (int64_t)b * a.count + j;
    a.out_scores[to] = -INFINITY;
    a.out_tokens[to] = a.out_parents[to] = -1;
    a.out_live[to] = 0;
  }
}

// Pieces: about four blocks a compute unit, and at least a step of each wave: 512 rows
// of 131072 fp16 words 31 us, with eight blocks a compute unit 35 and sixteen 41 (256 of
// 50257 fp32 words 16.6 and 6.4 to join, with seven blocks 18.0 and 7.0).
//
// At most kPieceMost words: a lane's 32-bit sum then takes eight parts of 32 terms
// (16 of 16 for fp32), and a row's sum is within 2^-16 of itself. In units of 2^-24,
// fp32 logits, 256 pieces: 20 additions of a lane, 45 where its maximum rises with each
// part (a product and an exponential of 1 ulp: 3), 15 in the wave and the block, 18 in
// the join, 2 of a term's own exponential, 2 of the logarithm, and the arguments'
// roundings, which along a term's way to the row's maximum add up to 2.23 times its
// distance t from it; the mean of t under the softmax is the entropy less the sum's
// logarithm, for 2^24 words at most 13.1. Together 131 (with 1024 pieces of four parts,
// too), and 90 for fp16, against 256.
constexpr int64_t kPieceMost = 65536;
struct Plan {
  int pieces, piece;
};
Plan plan(const BeamArgs& a) {
  const int64_t rows = (int64_t)a.batch * a.beams;
  const int64_t step = (int64_t)kWaves * kVectors * kWave * (a.fp32 ? 4 : 8);
  const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(rows, 1));
  int64_t piece = (a.vocab + want - 1) / want;
  piece = std::min(std::max((piece + step - 1) / step * step, step), kPieceMost);
  // (pieces of one length, since a step of few words takes as long: 32 rows of 16520 words
  // with 29 places 17.3 us, with a piece of 136 words after the others 22.3)
  const int64_t pieces = std::max<int64_t>((a.vocab + piece - 1) / piece, 1), wave = step / kWaves / kVectors;
  piece = std::max(((a.vocab + pieces - 1) / pieces + wave - 1) / wave * wave, wave);
  Plan p;
  p.piece = (int)piece;
  p.pieces = (int)((a.vocab + piece - 1) / piece);
  return p;
}

}  // namespace

size_t beam_workspace_bytes(const BeamArgs& a) {
  const Plan p = plan(a);
  return (size_t)a.batch * a.beams * p.pieces * (8 + 8 * (size_t)a.count);
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
  const Plan p = plan(a);
  const int64_t blocks = (int64_t)a.batch * a.beams * p.pieces;
  if (blocks > UINT32_MAX / kBlockThreads) return hipErrorInvalidValue;
  if (blocks > 0) {
    // (fewer words than 16 bytes hold: a kernel that does not load so many)
    const bool few = a.vocab < (a.fp32 ? 4 : 8);
    auto* const rows = a.fp32 ? few ? k_beam_rows<false, true> : k_beam_rows<false, false>
                              : few ? k_beam_rows<true, true> : k_beam_rows<true, false>;
    rows<<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, p.pieces, p.piece);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_beam_join<<<(uint32_t)a.batch, kJoinThreads, a.beams * 12, s>>>(a, p.pieces);
  return hipGetLastError();
}

}  // namespace i8mm
