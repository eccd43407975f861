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

#include "device_common.h"
#include "launchers.h"

namespace i8mm {

namespace {

constexpr int kWaves = kBlockThreads / kWave;
constexpr int kVectors = 4;   // 16-byte loads a lane takes at once
constexpr float kLog2E = 1.44269504088896340736f;

// 16 bytes of a row, which begins at any element.
struct __attribute__((packed, aligned(2))) Loose16 {
  v4i32 x;
};

// Whole-wave shift by one lane: lane l gets lane l - 1's (DPP wave_shr:1).
__device__ __forceinline__ uint32_t from_lane_below(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x138, 0xf, 0xf, false);
}
__device__ __forceinline__ float lane_float(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// The best of a row's piece, over the lanes of a wave: lane j holds the j-th.
// Equal values stand in the order of their index. Empty places hold -infinity and
// index 0, which nothing that is a candidate (more than -infinity) comes after.
struct Best {
  float v = -INFINITY;
  uint32_t i = 0;
  float last_v = -INFINITY;   // of place count - 1: what a candidate has to beat
  uint32_t last_i = 0;
  __device__ __forceinline__ bool takes(float x, uint32_t at) const {
    return x > last_v || (x == last_v && at < last_i);
  }
  // (uniform x and at that the list takes)
  __device__ __forceinline__ void insert(float x, uint32_t at, int lane, int count) {
    const int place = __popcll(__ballot(v > x || (v == x && i < at)));
    const float up = __builtin_bit_cast(float, from_lane_below(__builtin_bit_cast(uint32_t, v)));
    const uint32_t up_i = from_lane_below(i);
    v = lane < place ? v : lane == place ? x : up;
    i = lane < place ? i : lane == place ? at : up_i;
    last_v = lane_float(v, count - 1);
    last_i = (uint32_t)__builtin_amdgcn_readlane((int)i, count - 1);
  }
};

// A value that at least `count` lanes' x reach (-infinity where fewer are more
// than that), within 2^-7 of the largest such: the order of floats as integers,
// its upper 16 bits searched bit by bit.
__device__ __forceinline__ float reached_by(float x, int count) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const uint32_t key = (b ^ ((uint32_t)((int)b >> 31) | 0x80000000u)) >> 16;
  uint32_t t = 0;
#pragma unroll
  for (uint32_t bit = 0x8000u; bit; bit >>= 1)
    if (__popcll(__ballot(key >= (t | bit))) >= count) t |= bit;
  if (t <= 0x007fu) return -INFINITY;
  t <<= 16;
  return __builtin_bit_cast(float, t & 0x80000000u ? t ^ 0x80000000u : ~t);
}

// What a piece leaves: its maximum and sum, then `count` values and as many
// indices, best first.
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

// One block a piece. A wave takes 4 KB at a time; its first 4 KB set a floor for
// its list, what `count` of its lanes' maxima reach, so that the list starts with
// about `count` insertions.
template <bool kHalf>
__global__ __launch_bounds__(kBlockThreads) void k_beam_rows(BeamArgs a, int pieces, int piece) {
  constexpr int kV = kHalf ? 8 : 4, kStep = kVectors * kWave * kV;
  __shared__ float s_v[kWaves][kWave], s_m[kWaves], s_l[kWaves];
  __shared__ uint32_t s_i[kWaves][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = blockIdx.x / pieces, at_piece = blockIdx.x % pieces;
  if (a.live && a.live[row] == 0) return;   // the join reads nothing of it
  const int64_t begin = (int64_t)at_piece * piece;
  const int n = (int)min((int64_t)piece, a.vocab - begin);
  const uint16_t* const p16 = static_cast<const uint16_t*>(a.logits) + row * a.row_stride + begin;
  const float* const p32 = static_cast<const float*>(a.logits) + row * a.row_stride + begin;

  Best best;
  float m = -INFINITY, l = 0.f;
  for (int at = wave * kStep; at < n; at += kWaves * kStep) {
    float x[kVectors][kV], top[kVectors];
    int i0[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      i0[u] = at + (u * kWave + lane) * kV;
      if (i0[u] + kV <= n) {
        v4i32 t;
        if constexpr (kHalf) {
          t = reinterpret_cast<const Loose16*>(p16 + i0[u])->x;
#pragma unroll
          for (int e = 0; e < kV; ++e)
            x[u][e] = h2f(((uint32_t)t[e >> 1] >> (16 * (e & 1))) & 0xffffu);
        } else {
          t = reinterpret_cast<const Loose16*>(p32 + i0[u])->x;
#pragma unroll
          for (int e = 0; e < kV; ++e) x[u][e] = __builtin_bit_cast(float, (uint32_t)t[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kV; ++e)
          x[u][e] = i0[u] + e >= n ? -INFINITY : kHalf ? h2f(p16[i0[u] + e]) : p32[i0[u] + e];
      }
    }
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      top[u] = x[u][0];
#pragma unroll
      for (int e = 1; e < kV; ++e) top[u] = fmaxf(top[u], x[u][e]);
    }
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    // A NaN or +infinity makes the sum NaN, and the row one without candidates.
    const float next = fmaxf(m, most), base = next == -INFINITY ? 0.f : next;
    l *= __builtin_amdgcn_exp2f((m - base) * kLog2E);
    float sum[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      sum[u] = 0.f;
#pragma unroll
      for (int e = 0; e < kV; ++e) sum[u] += __builtin_amdgcn_exp2f((x[u][e] - base) * kLog2E);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    m = next;

    const float floor = at == wave * kStep ? reached_by(most, a.count) : -INFINITY;
    if (!__any(most >= floor && best.takes(most, (uint32_t)i0[0]))) continue;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      if (!__any(top[u] >= floor && best.takes(top[u], (uint32_t)i0[u]))) continue;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const uint32_t mine = (uint32_t)(i0[u] + e);
        uint64_t those = __ballot(x[u][e] >= floor && best.takes(x[u][e], mine));
        while (those) {
          const int from = __builtin_ctzll(those);
          those &= those - 1;
          const float v = lane_float(x[u][e], from);
          const uint32_t i = (uint32_t)__builtin_amdgcn_readlane((int)mine, from);
          if (best.takes(v, i)) best.insert(v, i, lane, a.count);
        }
      }
    }
  }

  // the wave's sum, then the block's
  float top = m;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  const float base = top == -INFINITY ? 0.f : top;
  l *= __builtin_amdgcn_exp2f((m - base) * kLog2E);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) l += __shfl_xor(l, d, kWave);
  s_v[wave][lane] = best.v;
  s_i[wave][lane] = best.i;
  if (lane == 0) {
    s_m[wave] = top;
    s_l[wave] = l;
  }
  __syncthreads();
  // An entry's place is the number of entries before it.
  const Pieces out = pieces_of(a.ws, (int64_t)a.batch * a.beams, pieces, a.count);
  const int64_t part = (int64_t)row * pieces + at_piece;
  const int entries = kWaves * a.count;
  if ((int)threadIdx.x < entries) {
    const int w = threadIdx.x / a.count, j = threadIdx.x % a.count;
    const float v = s_v[w][j];
    const uint32_t i = s_i[w][j];
    int place = j;
    for (int o = 0; o < kWaves; ++o) {
      if (o == w) continue;
      for (int k = 0; k < a.count; ++k) {
        const float ov = s_v[o][k];
        // (empty places are equal: those of earlier waves come first)
        place += ov > v || (ov == v && (s_i[o][k] < i || (s_i[o][k] == i && o < w)));
      }
    }
    if (place < a.count) {
      out.value[part * a.count + place] = v;
      out.index[part * a.count + place] = i + (uint32_t)begin;
    }
  }
  if (threadIdx.x == 0) {
    float t = s_m[0], sum = 0.f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t = fmaxf(t, s_m[w]);
    const float b = t == -INFINITY ? 0.f : t;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += s_l[w] * __builtin_amdgcn_exp2f((s_m[w] - b) * kLog2E);
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

// One block a search.
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave;
__global__ __launch_bounds__(kJoinThreads) void k_beam_join(BeamArgs a, int pieces) {
  extern __shared__ double s_base[];   // [beams]: what a beam's logits are added to
  __shared__ double s_v[kJoinWaves][kWave];
  __shared__ int64_t s_at[kJoinWaves][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x;
  const Pieces in = pieces_of(a.ws, (int64_t)a.batch * a.beams, pieces, a.count);
  for (int i = wave; i < a.beams; i += kJoinWaves) {
    const int64_t row = (int64_t)b * a.beams + i;
    const float s = a.scores[row];
    const double score = fabsf(s) < INFINITY ? (double)s : no_value();
    if (a.live && a.live[row] == 0) {
      if (lane == 0) s_base[i] = score;
      continue;
    }
    float top = -INFINITY;
    bool nan = false;
    for (int p = lane; p < pieces; p += kWave) {
      const float2 s = in.sum[row * pieces + p];
      top = fmaxf(top, s.x);
      nan |= !(s.y >= 0.f);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    double sum = 0.0;
    for (int p = lane; p < pieces; p += kWave) {
      const float2 s = in.sum[row * pieces + p];
      if (s.y > 0.f) sum += (double)s.y * exp((double)s.x - (double)top);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
    const bool empty = __any(nan) || !(top > -INFINITY);
    if (lane == 0) s_base[i] = empty ? no_value() : score - (double)top - log(sum);
  }
  __syncthreads();

  const double none = no_value();
  double best = none, last = none;   // as in the rows' lists
  int64_t best_at = 0, last_at = 0;
  // (no words: a beam that has ended still has its one candidate)
  const int per_beam = max(pieces * a.count, 1), all = a.beams * per_beam;
  const int64_t words = max(a.vocab, (int64_t)1);
  for (int e0 = wave * kWave; e0 < all; e0 += kJoinThreads) {
    double v = none;
    int64_t at = 0;
    const int e = e0 + lane, i = e / per_beam, k = e % per_beam;
    if (e < all) {
      const int64_t row = (int64_t)b * a.beams + i;
      if (a.live && a.live[row] == 0) {
        if (k == 0) {
          v = s_base[i];
          at = i * words + max(a.eos, 0);
        }
      } else if (s_base[i] > none) {
        v = s_base[i] + (double)in.value[row * per_beam + k];
        at = i * words + in.index[row * per_beam + k];
      }
    }
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
  s_v[wave][lane] = best;
  s_at[wave][lane] = best_at;
  __syncthreads();
  for (int e = threadIdx.x; e < kJoinWaves * a.count; e += kJoinThreads) {
    const int w = e / a.count, j = e % a.count;
    const double v = s_v[w][j];
    const int64_t at = s_at[w][j];
    int place = j;
    for (int o = 0; o < kJoinWaves; ++o) {
      if (o == w) continue;
      for (int k = 0; k < a.count; ++k) {
        const double ov = s_v[o][k];
        const int64_t o_at = s_at[o][k];
        // (empty places are equal: those of earlier waves come first)
        place += before(ov, o_at, v, at) || (ov == v && o_at == at && o < w);
      }
    }
    if (place >= a.count) continue;
    const bool found = v > none;
    const int64_t i = at / words;
    const int64_t to = (int64_t)b * a.count + place;
    const int64_t row = (int64_t)b * a.beams + i;
    const bool ended = a.live && a.live[row] == 0;
    const int token = ended ? a.eos : (int)(at - i * words);
    a.out_scores[to] = (float)v;
    a.out_tokens[to] = found ? token : -1;
    a.out_parents[to] = found ? (int)row : -1;
    a.out_live[to] = found && token != a.eos;
  }
}

// Pieces: about four blocks a compute unit, and at least a step of each wave. At
// most kPieceMost words: a lane's 32-bit sum then takes eight parts of 32 terms
// (16 of 16 for fp32), which keeps its error below 2^-18: 10 and 16 roundings of
// sums, as many of rescaling, the exponential's 2^-23, and its argument's, 2^-24 of
// itself, which terms that matter have below the logarithm of their number.
constexpr int64_t kPieceMost = 65536;
struct Plan {
  int pieces, piece;
};
Plan plan(const BeamArgs& a) {
  const int64_t rows = (int64_t)a.batch * a.beams;
  const int64_t step = (int64_t)kWaves * kVectors * kWave * (a.fp32 ? 4 : 8);
  const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(rows, 1));
  int64_t piece = (a.vocab + want - 1) / want;
  piece = std::max((piece + step - 1) / step * step, step);
  Plan p;
  p.piece = (int)std::min(piece, kPieceMost);
  p.pieces = (int)((a.vocab + p.piece - 1) / p.piece);
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
  if (blocks > INT32_MAX / kBlockThreads) return hipErrorInvalidValue;
  if (blocks > 0) {
    if (a.fp32)
      k_beam_rows<false><<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, p.pieces, p.piece);
    else
      k_beam_rows<true><<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, p.pieces, p.piece);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_beam_join<<<(uint32_t)a.batch, kJoinThreads, a.beams * sizeof(double), s>>>(a, p.pieces);
  return hipGetLastError();
}

}  // namespace i8mm
