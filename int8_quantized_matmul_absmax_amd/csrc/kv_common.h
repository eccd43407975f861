// Device helpers shared by the kernels of the paged 8-bit key/value cache.
#pragma once

#include "device_common.h"
#include "launchers.h"

namespace i8mm {

constexpr int kKvBlock = I8MM_KV_BLOCK;   // tokens of a block
constexpr int kTile = 256;                // bytes of a 16 x 16 code tile

// What the kernels take from a sequence's entries, bounded as the header
// says, so that no content of the arrays reaches past a buffer: new tokens
// are positions [first, len) (first < 0 for tokens before the sequence), rows
// row0 .. row0 + n - 1 of the packed tensors. The rows after them up to `stop`
// belong to no sequence: tokens beyond max_tokens and, after the last sequence,
// the rest.
struct KvSeq {
  int row0, n, len, first, stop;
};
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int b) {
  KvSeq s;
  int lo = b, hi = b + 1;
  if (a.cu_tokens) {
    lo = min(max(a.cu_tokens[b], 0), a.total_tokens);
    hi = min(max(a.cu_tokens[b + 1], lo), a.total_tokens);
  }
  s.row0 = lo;
  s.n = min(hi - lo, a.max_tokens);
  s.len = min(max(a.seq_lens[b], 0), a.len_cap);
  s.first = s.len - s.n;
  s.stop = a.cu_tokens && b == a.num_seqs - 1 ? a.total_tokens : hi;
  return s;
}

__device__ __forceinline__ int page_or_none(const KvArgs& a, int page) {
  return (uint32_t)page < (uint32_t)a.num_pages ? page : -1;
}

// A wave writes zeros to `bytes` (a multiple of 16).
__device__ __forceinline__ void zero_bytes(void* p, int bytes, int lane) {
  for (int i = lane * 16; i < bytes; i += kWave * 16)
    *reinterpret_cast<v4i32*>(static_cast<int8_t*>(p) + i) = v4i32{0, 0, 0, 0};
}

// Number of block `blk` (16 tokens) of sequence b for head h among all blocks
// of the cache, or -1 when its page is absent. blk >= 0 and below the
// sequence's blocks.
__device__ __forceinline__ int kv_block(const KvArgs& a, int b, int h, int blk) {
  const uint32_t pg = (uint32_t)blk / (uint32_t)a.slots;
  const int page = a.page_table[(int64_t)b * a.max_pages + pg];
  if ((uint32_t)page >= (uint32_t)a.num_pages) return -1;
  return (page * a.kv_heads + h) * a.slots + (blk - (int)pg * a.slots);
}

// 16 bytes as a vector type (the struct uint4 keeps values of branches in
// memory, and loads of it without a type for alias analysis).
__device__ __forceinline__ v4i32 ld16v(const void* p) { return *reinterpret_cast<const v4i32*>(p); }
__device__ __forceinline__ v4f32 ld16f(const float* p) { return *reinterpret_cast<const v4f32*>(p); }

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

__device__ __forceinline__ void unpack8(const v4i32& t, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = h2f(((uint32_t)t[e >> 1] >> (16 * (e & 1))) & 0xffffu);
}

// The rotation of 8 features, one rounding an operation, in the order the
// header states. rotate_pairs: four pairs of neighbours. rotate_half: x are
// eight first (low) or second members of pairs, other their partners.
__device__ __forceinline__ void rotate_pairs(const v4f32& c, const v4f32& s, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = a * c[i] - b * s[i];
    x[2 * i + 1] = b * c[i] + a * s[i];
  }
}
__device__ __forceinline__ void rotate_half(const v4f32& c0, const v4f32& c1, const v4f32& s0,
                                            const v4f32& s1, const float* other, bool low,
                                            float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float own = x[i] * (i < 4 ? c0[i & 3] : c1[i & 3]);
    const float far = other[i] * (i < 4 ? s0[i & 3] : s1[i & 3]);
    x[i] = low ? own - far : own + far;
  }
}

// The sequence whose rows token t is among: the last that begins at t or before.
// 64 probes at once.
__device__ __forceinline__ int sequence_of(const KvArgs& a, int t, int lane) {
  if (!a.cu_tokens) return t;
  int b = 0;
  for (int size = a.num_seqs; size > 0;) {
    const int step = (size + kWave - 1) / kWave, ahead = lane * step;
    const bool before = ahead < size && a.cu_tokens[b + ahead] <= t;
    const int n = __popcll(__ballot(before));
    if (n == 0) break;
    const int at = (n - 1) * step;
    b += at;
    size = step == 1 ? 0 : min(step, size - at);
  }
  return b;
}

// Exclusive prefix sum over the block's kWaves waves, and the total. Two barriers.
template <int kWaves>
__device__ __forceinline__ int block_prefix(int v, int* s_wave, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int incl = wave_inclusive_scan_dpp(v);
  if (lane == 63) s_wave[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int s = s_wave[w];
    before += w < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

#define I8MM_KV_DIMS(D, CALL) \
  switch (D) {                \
    case 64: { CALL(64); } break;   \
    case 80: { CALL(80); } break;   \
    case 96: { CALL(96); } break;   \
    case 128: { CALL(128); } break; \
    default: { CALL(256); } break;  \
  }

}  // namespace i8mm
