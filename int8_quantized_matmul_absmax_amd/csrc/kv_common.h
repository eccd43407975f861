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
// row0 .. row0 + n - 1 of the packed tensors.
struct KvSeq {
  int row0, n, len, first;
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
  return s;
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

__device__ __forceinline__ void unpack8(const uint4& t, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = h2f(half_of(t, e));
}

// Features e0 .. e0 + 7 of a head's row `p` in fp32, rotated for position pos
// when they lie in the rotated part (r.cos set, e0 < r.dim). r.dim is a
// multiple of 16, so a group of 8 lies on one side of r.dim / 2 and of r.dim.
// One rounding an operation, in the order the header states.
__device__ __forceinline__ void load8_rotated(const uint16_t* p, int e0, int pos,
                                              const RotaryArgs& r, float* x) {
  unpack8(ld16(p + e0), x);
  if (!r.cos || e0 >= r.dim) return;
  const int half = r.dim >> 1;
  const int64_t row = (int64_t)pos * half;
  if (r.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(r.cos + row + (e0 >> 1));
    const float4 s = *reinterpret_cast<const float4*>(r.sin + row + (e0 >> 1));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cc[i] - b * ss[i];
      x[2 * i + 1] = b * cc[i] + a * ss[i];
    }
    return;
  }
  const bool low = e0 < half;
  const int i0 = low ? e0 : e0 - half;
  float y[8];
  unpack8(ld16(p + (low ? e0 + half : e0 - half)), y);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 c = *reinterpret_cast<const float4*>(r.cos + row + i0 + 4 * u);
    const float4 s = *reinterpret_cast<const float4*>(r.sin + row + i0 + 4 * u);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float own = x[4 * u + i] * cc[i], other = y[4 * u + i] * ss[i];
      x[4 * u + i] = low ? own - other : own + other;
    }
  }
}

}  // namespace i8mm
