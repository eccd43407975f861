// Append to and read from the paged 8-bit key/value cache.
//
// Both move one block of 16 tokens and one head a wave, keys and values apart.
// Keys: codes of a token lie along the features, so lanes hold 8 features of a
// token. Values: codes of a feature lie along the tokens, so a lane holds a
// pair of features for all 16 tokens, and the transposition costs no exchange.
//
// Both are bound by memory: for 4096 tokens of 96 heads of 128 features append
// moves 302 MB in 66 us (4.6 TB/s) and read as much in 49 us; reading 59500
// tokens of 16 heads of 128 back (731 MB) takes 158 us, 4.6 TB/s, where a large copy
// moves 5.2. With few tokens a launch is what they cost (5 to 6 us of latency: the
// batch's arrays, the page table, then the block).

#include "kv_common.h"

namespace i8mm {

namespace {

// New keys and values are read once, and values read back are written once:
// streaming accesses (for 4096 tokens of 96 heads of 128 append takes 66 us, 74 us
// with plain ones, and reading the new codes back 49 us against 75).
template <class T>
__device__ __forceinline__ T ld_once(const T* p) { return __builtin_nontemporal_load(p); }
template <class T>
__device__ __forceinline__ void st_once(T* p, T x) { __builtin_nontemporal_store(x, p); }

// Absmaxes up to 2^-119 count as 0 (127 / a stays finite above it).
constexpr uint32_t kTinyAbsmax = 0x04000000u;

__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// Low byte: the code rne(y), abs(y) <= 127 up to one rounding.
__device__ __forceinline__ uint32_t code_bits(float y) {
  return __builtin_bit_cast(uint32_t, y + 12582912.0f);
}
__device__ __forceinline__ float byte_code(uint32_t w, int i) {
  return (float)(int8_t)(w >> (8 * i));
}
// Four old codes over a larger absmax.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  return pack4(code_bits(byte_code(w, 0) * ratio), code_bits(byte_code(w, 1) * ratio),
               code_bits(byte_code(w, 2) * ratio), code_bits(byte_code(w, 3) * ratio));
}

struct BlockScale {
  float s, ratio, a;
  bool grown;   // the old codes change
};
// The block's absmax after the append from the bit patterns of the old one
// and of the new elements' (unsigned order: NaN above infinity above finite).
__device__ __forceinline__ BlockScale block_scale(uint32_t a_old, uint32_t a_new) {
  uint32_t a = a_old > a_new ? a_old : a_new;
  if (a <= kTinyAbsmax) a = 0;
  BlockScale r;
  r.a = __builtin_bit_cast(float, a);
  r.s = a ? 127.0f / r.a : 0.f;
  r.ratio = a ? __builtin_bit_cast(float, a_old) / r.a : 0.f;
  r.grown = a != a_old;
  return r;
}

// One block of 16 tokens of `heads` heads from head h0 on. Rows [0, r0) of the
// block are older tokens, [r0, r1) new ones, src0 the packed row of row 0 (which
// need not exist), t0 its position.
struct NewRows {
  int b, blk, h0, heads, r0, r1, t0;
  int64_t src0;
};

// Lanes hold 8 features of a token. The rotation's factors are the same for
// every head and loaded once.
template <int D>
__device__ __forceinline__ void append_keys(const uint16_t* __restrict__ k, int64_t ts, int64_t hs,
                                            const KvArgs& a, const RotaryArgs& rot,
                                            const NewRows& w, int lane) {
  constexpr int kChunks = D / 8, kItems = kKvBlock * kChunks;
  constexpr int kIter = (kItems + kWave - 1) / kWave;
  const int half = rot.dim >> 1;
  v4f32 cos[kIter][2], sin[kIter][2];
  if (rot.cos) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int idx = it * kWave + lane, tok = min(max(idx / kChunks, w.r0), w.r1 - 1);
      const int e0 = idx % kChunks * 8, e = e0 < rot.dim ? e0 : 0;
      const int i0 = rot.interleaved ? e >> 1 : e < half ? e : e - half;
      const int64_t at = (int64_t)(w.t0 + tok) * half + i0;
      const int more = rot.interleaved ? 0 : 4;
      cos[it][0] = ld16f(rot.cos + at);
      cos[it][1] = ld16f(rot.cos + at + more);
      sin[it][0] = ld16f(rot.sin + at);
      sin[it][1] = ld16f(rot.sin + at + more);
    }
  }
  for (int h = w.h0; h < w.h0 + w.heads; ++h) {
    const uint16_t* src = k + (int64_t)h * hs;
    v4i32 own[kIter], other[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int idx = it * kWave + lane, tok = min(max(idx / kChunks, w.r0), w.r1 - 1);
      const int e0 = idx % kChunks * 8, e = e0 < rot.dim ? e0 : 0;
      const uint16_t* row = src + (w.src0 + tok) * ts;
      own[it] = ld_once(reinterpret_cast<const v4i32*>(row + e0));
      if (rot.cos && !rot.interleaved) other[it] = ld16v(row + (e < half ? e + half : e - half));
    }
    const int lin = kv_block(a, w.b, h, w.blk);
    if (lin < 0) continue;
    int8_t* tile = a.k_codes + (int64_t)lin * (kKvBlock * D);
    const uint32_t a_old = w.r0 > 0 ? abs_bits(a.k_absmax[lin]) : 0u;
    float x[kIter][8];
    uint32_t top = 0;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int idx = it * kWave + lane, tok = idx / kChunks, e0 = idx % kChunks * 8;
      unpack8(own[it], x[it]);
      if (rot.cos && e0 < rot.dim) {
        if (rot.interleaved) {
          rotate_pairs(cos[it][0], sin[it][0], x[it]);
        } else {
          float far[8];
          unpack8(other[it], far);
          rotate_half(cos[it][0], cos[it][1], sin[it][0], sin[it][1], far, e0 < half, x[it]);
        }
      }
      const bool live = tok >= w.r0 && tok < w.r1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[it][e] = live ? x[it][e] : 0.f;
        const uint32_t m = abs_bits(x[it][e]);
        top = top > m ? top : m;
      }
    }
    const BlockScale sc = block_scale(a_old, wave_max_u32_dpp(top));
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int idx = it * kWave + lane, tok = idx / kChunks, e0 = idx % kChunks * 8;
      if (idx >= kItems) continue;
      uint2* dst = reinterpret_cast<uint2*>(tile + (e0 >> 4) * kTile + tok * 16 + (e0 & 15));
      if (tok < w.r0) {
        if (!sc.grown) continue;
        const uint2 o = *dst;
        *dst = make_uint2(rescale4(o.x, sc.ratio), rescale4(o.y, sc.ratio));
      } else {
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = code_bits(x[it][e] * sc.s);
        *dst = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
      }
    }
    if (lane == 0) a.k_absmax[lin] = sc.a;
  }
}

// A lane holds a pair of features for all 16 tokens.
template <int D>
__device__ __forceinline__ void append_values(const uint16_t* __restrict__ v, int64_t ts,
                                              int64_t hs, const KvArgs& a, const NewRows& w,
                                              int lane) {
  constexpr int kPairs = D / 2, kIter = (kPairs + kWave - 1) / kWave;
  for (int h = w.h0; h < w.h0 + w.heads; ++h) {
    uint32_t x[kIter][kKvBlock];   // pairs of fp16
    uint32_t top = 0;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int p = it * kWave + lane;
#pragma unroll
      for (int r = 0; r < kKvBlock; ++r) {
        x[it][r] = 0;
        if (r >= w.r0 && r < w.r1 && p < kPairs)
          x[it][r] = ld_once(reinterpret_cast<const uint32_t*>(v + (w.src0 + r) * ts + h * hs + 2 * p));
      }
    }
    const int lin = kv_block(a, w.b, h, w.blk);
    if (lin < 0) continue;
    int8_t* tile = a.v_codes + (int64_t)lin * (kKvBlock * D);
    const uint32_t a_old = w.r0 > 0 ? abs_bits(a.v_absmax[lin]) : 0u;
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int r = 0; r < kKvBlock; ++r) {
        const uint32_t lo = x[it][r] & 0x7fffu, hi = (x[it][r] >> 16) & 0x7fffu;
        const uint32_t m = lo > hi ? lo : hi;   // fp16 patterns order as their magnitudes
        top = top > m ? top : m;
      }
    const BlockScale sc = block_scale(a_old, abs_bits(h2f(wave_max_u32_dpp(top))));
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int p = it * kWave + lane;
      if (p >= kPairs) continue;
      // the pair's two features are 32 consecutive bytes
      uint4* dst = reinterpret_cast<uint4*>(tile + p * 32);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t c4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[i] = code_bits(h2f((x[it][4 * q + i] >> (16 * f)) & 0xffffu) * sc.s);
          c4[q] = pack4(c[0], c[1], c[2], c[3]);
        }
        if (w.r0 > 0) {
          const uint4 o = dst[f];
          const uint32_t old[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int rows = min(max(w.r0 - 4 * q, 0), 4);   // old rows among these four
            const uint32_t keep = rows >= 4 ? 0xffffffffu : (1u << (8 * rows)) - 1u;
            const uint32_t ow = sc.grown ? rescale4(old[q], sc.ratio) : old[q];
            c4[q] = (ow & keep) | (c4[q] & ~keep);
          }
        }
        dst[f] = make_uint4(c4[0], c4[1], c4[2], c4[3]);
      }
    }
    if (lane == 0) a.v_absmax[lin] = sc.a;
  }
}

// A wave takes a block's keys or values for `per_wave` heads.
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_append(
    const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs, const uint16_t* __restrict__ v,
    int64_t v_ts, int64_t v_hs, KvArgs a, RotaryArgs rot, int tasks, int per_wave) {
  const int lane = threadIdx.x & 63;
  const int task = blockIdx.x * (kBlockThreads / kWave) +
                   __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= tasks) return;
  const int parts = (a.kv_heads + per_wave - 1) / per_wave, part = (task >> 1) % parts;
  NewRows w;
  w.b = blockIdx.y;
  const KvSeq sq = kv_seq(a, w.b);
  w.blk = max(sq.first, 0) / kKvBlock + (task >> 1) / parts;
  w.t0 = w.blk * kKvBlock;
  if (sq.n <= 0 || w.t0 >= sq.len) return;
  w.h0 = part * per_wave;
  w.heads = min(per_wave, a.kv_heads - w.h0);
  w.r0 = max(sq.first - w.t0, 0);
  w.r1 = min(kKvBlock, sq.len - w.t0);
  w.src0 = (int64_t)sq.row0 + w.t0 - sq.first;
  if (task & 1)
    append_values<D>(v, v_ts, v_hs, a, w, lane);
  else
    append_keys<D>(k, k_ts, k_hs, a, rot, w, lane);
}

template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_read(KvArgs a, uint16_t* __restrict__ k,
                                                           uint16_t* __restrict__ v, int tasks) {
  const int lane = threadIdx.x & 63;
  const int task = blockIdx.x * (kBlockThreads / kWave) + (threadIdx.x >> 6);
  const int b = blockIdx.y;
  if (task >= tasks) return;
  const bool values = task & 1;
  uint16_t* out = values ? v : k;
  if (!out) return;
  const int h = (task >> 1) % a.kv_heads;
  const KvSeq sq = kv_seq(a, b);
  if (__builtin_expect(sq.row0 + sq.n < sq.stop, 0))   // (0.6% of a large read when not marked)
    for (int64_t r = (int64_t)sq.row0 + sq.n + (task >> 1); r < sq.stop; r += tasks >> 1)
      zero_bytes(out + r * a.kv_heads * D, 2 * a.kv_heads * D, lane);
  // floor division: a sequence with n > len starts at a negative position
  const int blk = (sq.first >> 4) + (task >> 1) / a.kv_heads;
  const int t0 = blk * kKvBlock;
  if (sq.n <= 0 || t0 >= sq.len) return;
  const int r0 = max(sq.first - t0, 0), r1 = min(kKvBlock, sq.len - t0);
  const int lin = blk >= 0 ? kv_block(a, b, h, blk) : -1;
  const int64_t ts = (int64_t)a.kv_heads * D;
  uint16_t* dst0 = out + ((int64_t)sq.row0 + t0 - sq.first) * ts + (int64_t)h * D;

  if (!values) {
    constexpr int kTiles = D / 16, kItems = kKvBlock * kTiles;
    constexpr int kIter = (kItems + kWave - 1) / kWave;
    const float step = lin >= 0 ? a.k_absmax[lin] / 127.0f : 0.f;
    const int8_t* tile = a.k_codes + (int64_t)lin * (kKvBlock * D);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int idx = it * kWave + lane, tok = idx / kTiles, c = idx % kTiles;
      if (tok < r0 || tok >= r1) continue;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (lin >= 0) w = ld16(tile + c * kTile + tok * 16);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = f2h2(byte_code(ww[i >> 1], (2 * i) & 3) * step,
                    byte_code(ww[i >> 1], (2 * i + 1) & 3) * step);
      uint16_t* dst = dst0 + tok * ts + c * 16;
      st_once(reinterpret_cast<v4i32*>(dst), v4i32{(int)o[0], (int)o[1], (int)o[2], (int)o[3]});
      st_once(reinterpret_cast<v4i32*>(dst + 8), v4i32{(int)o[4], (int)o[5], (int)o[6], (int)o[7]});
    }
    return;
  }
  constexpr int kPairs = D / 2, kIter = (kPairs + kWave - 1) / kWave;
  const float step = lin >= 0 ? a.v_absmax[lin] / 127.0f : 0.f;
  const int8_t* tile = a.v_codes + (int64_t)lin * (kKvBlock * D);
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int p = it * kWave + lane;
    if (p >= kPairs) continue;
    uint4 f0 = make_uint4(0, 0, 0, 0), f1 = f0;
    if (lin >= 0) {
      f0 = ld16(tile + p * 32);
      f1 = ld16(tile + p * 32 + 16);
    }
    const uint32_t w0[4] = {f0.x, f0.y, f0.z, f0.w}, w1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
    for (int r = 0; r < kKvBlock; ++r)
      if (r >= r0 && r < r1)
        st_once(reinterpret_cast<uint32_t*>(dst0 + r * ts + 2 * p),
                f2h2(byte_code(w0[r >> 2], r & 3) * step, byte_code(w1[r >> 2], r & 3) * step));
  }
}

// Blocks that the new tokens of one sequence can touch.
int64_t max_blocks(const KvArgs& a) { return ((int64_t)a.max_tokens + 2 * kKvBlock - 2) / kKvBlock; }

}  // namespace

bool kv_head_dim_ok(int64_t D) { return D == 64 || D == 80 || D == 96 || D == 128 || D == 256; }

hipError_t launch_kv_append(const uint16_t* k, int64_t k_ts, int64_t k_hs, const uint16_t* v,
                            int64_t v_ts, int64_t v_hs, const KvArgs& a, const RotaryArgs& r,
                            hipStream_t s) {
  // Four heads a wave once there are waves enough: they share the rotation's
  // factors (4096 tokens of 96 heads of 128: 66 us, with one 83). With few tokens
  // the heads are what there is to run at once (16 tokens of 32 heads: 5.8 us with
  // one, with four 13). At 8256 waves, 2048 tokens of 32 heads, four take 18.0 us and
  // one 20.5 (64 features 14.2 and 15.5, 256 38 and 50), at 4160 15.2 and 13.7 (12.4
  // and 10.1, 22.5 and 27.9).
  const int64_t one = max_blocks(a) * a.kv_heads * 2 * a.num_seqs;
  const int per_wave = one >= 8192 ? 4 : 1;
  const int64_t parts = (a.kv_heads + per_wave - 1) / per_wave;
  const int64_t tasks = max_blocks(a) * parts * 2;
  if (tasks > INT32_MAX - 4) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)((tasks + 3) / 4), (uint32_t)a.num_seqs);
#define CALL(D)                                                                                  \
  k_kv_append<D><<<grid, kBlockThreads, 0, s>>>(k, k_ts, k_hs, v, v_ts, v_hs, a, r, (int)tasks, \
                                                per_wave)
  I8MM_KV_DIMS(a.head_dim, CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs& a, uint16_t* k, uint16_t* v, hipStream_t s) {
  const int64_t tasks = max_blocks(a) * a.kv_heads * 2;
  if (tasks > INT32_MAX - 4) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)((tasks + 3) / 4), (uint32_t)a.num_seqs);
#define CALL(D) k_kv_read<D><<<grid, kBlockThreads, 0, s>>>(a, k, v, (int)tasks)
  I8MM_KV_DIMS(a.head_dim, CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace i8mm
