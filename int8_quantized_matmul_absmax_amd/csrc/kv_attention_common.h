// What the attention kernels over the paged 8-bit key/value cache share: queries
// as 15-bit integers, the staging of codes, the scores and weights of a group, and
// the join of a row's splits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "kv_common.h"

namespace i8mm {

namespace {

constexpr int kGroup = 64;          // tokens of a step: four blocks
constexpr int kRows = 16;           // rows of a tile
constexpr float kHead = 7.f;        // of m below a row's maximum
constexpr float kLazy = 8.f;        // a row is rescaled when its maximum grew by more
constexpr float kMinAbsmax = 0x1p-40f;   // of values

// The workspace of a launch with several splits: for each split and row the sum
// O (of codes, not divided) and its maximum and row sum, and for each row the number of
// splits that see some of it, written by the first.
struct Parts {
  float* o;        // [splits][rows][D]
  float* ml;       // [splits][rows][2]
  int32_t* count;  // [rows]
  int64_t rows;
};
__host__ __device__ __forceinline__ Parts parts_of(float* ws, int64_t rows, int splits, int D) {
  Parts p;
  p.o = ws;
  p.ml = ws + splits * rows * D;
  p.count = reinterpret_cast<int32_t*>(p.ml + splits * rows * 2);
  p.rows = rows;
  return p;
}

// Maximum over the lanes that share a row: l ^ 32, and with four also l ^ 16.
template <int kLanes>
__device__ __forceinline__ float max_over_groups(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
  if constexpr (kLanes == 4) {
    u = __builtin_bit_cast(uint32_t, v);
    const auto q = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)q[0]), __builtin_bit_cast(float, (uint32_t)q[1]));
  }
  return v;
}

// 16 codes as fp16: 0x6400 | (code + 128) is 1152 + code.
__device__ __forceinline__ void codes_to_f16(const v4i32& w, v8f16* lo, v8f16* hi) {
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (uint32_t)w[i] ^ 0x80808080u;
    out[2 * i] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
    out[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
  }
  const v2f16 off = {(_Float16)-1152.f, (_Float16)-1152.f};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    out[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2f16, out[i]) + off);
  *lo = __builtin_bit_cast(v8f16, make_uint4(out[0], out[1], out[2], out[3]));
  *hi = __builtin_bit_cast(v8f16, make_uint4(out[4], out[5], out[6], out[7]));
}

// LDS stores written as the instruction itself: before a plain store the
// compiler waits for every copy into LDS in flight, which these never meet. A
// wave's own reads come after them in order; for other waves, the barrier in
// between waits for them.
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef int32_t v2i32 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void lds_store(int8_t* p, v4i32 x) {
  asm volatile("ds_write_b128 %0, %1" : : "v"((uint32_t)(uintptr_t)(lds_ptr_t)p), "v"(x) : "memory");
}
__device__ __forceinline__ void lds_store(int8_t* p, v2i32 x) {
  asm volatile("ds_write_b64 %0, %1" : : "v"((uint32_t)(uintptr_t)(lds_ptr_t)p), "v"(x) : "memory");
}
__device__ __forceinline__ void lds_store(float* p, float x) {
  asm volatile("ds_write_b32 %0, %1" : : "v"((uint32_t)(uintptr_t)(lds_ptr_t)p), "v"(x) : "memory");
}

// Queries into LDS as the products take them: per row kC * 64 bytes of hi, then
// as many of lo, zero past D, and q's factor a / 16256. Lanes lie along the rows,
// so that features and rotation factors are read in whole lines (read as
// operands, 16 rows an instruction, they cost each block 15 us), and a lane has
// twice eight features: of the rotated ones eight and their partners (or, for
// pairs of neighbours, eight of each half), of the rest sixteen in a row.
// Loads and what is made of them are apart, so that every load is on its way
// before the first is waited for; and without branches: features that are not
// rotated load factors that are not used (the first ones', or with no rotation at
// all `some` memory's) and take cos 1, sin 0.
template <int D>
struct QueryCfg {
  static constexpr int kC = (D + 63) / 64;
  static constexpr int kLanes = 4 * kC;                 // of a row
  static constexpr int kPassRows = kWave / kLanes;
  static constexpr int kRowBytes = 2 * 64 * kC;
};
struct QueryLoads {
  v4i32 x[2];
  v4f32 cos[2], sin[2];
};
// Where a lane's two runs of eight features lie; whether they are rotated.
template <int D>
__device__ __forceinline__ bool query_features(const RotaryArgs& rot, int lane, int (&e)[2]) {
  const int u = lane % QueryCfg<D>::kLanes;
  const bool rotated = 16 * u < rot.dim;
  e[0] = rotated ? 8 * u : 16 * u;
  e[1] = e[0] + (rotated ? rot.dim >> 1 : 8);
  return rotated;
}
template <int D>
__device__ __forceinline__ void load_query(const uint16_t* row, int pos, const RotaryArgs& rot,
                                           const void* some, int lane, QueryLoads& in) {
  int e[2];
  const bool rotated = query_features<D>(rot, lane, e);
  const int64_t at = rot.cos ? (int64_t)pos * (rot.dim >> 1) : 0;
  const float* cos = (rot.cos ? rot.cos : static_cast<const float*>(some)) + at;
  const float* sin = (rot.cos ? rot.sin : static_cast<const float*>(some)) + at;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int i = !rotated ? 0 : rot.interleaved ? e[w] >> 1 : e[0] + 4 * w;
    in.x[w] = ld16v(row + min(e[w], D - 8));
    in.cos[w] = ld16f(cos + i);
    in.sin[w] = ld16f(sin + i);
  }
}
// A lane's rotated part of the row, and its absmax's bit pattern.
template <int D>
__device__ __forceinline__ uint32_t rotate_query(const QueryLoads& in, bool live,
                                                 const RotaryArgs& rot, int lane, float (&x)[16]) {
  int e[2];
  const bool rotated = query_features<D>(rot, lane, e);
  const int keep = live && e[0] < D ? -1 : 0;
  v4f32 cs[2], sn[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    unpack8(in.x[w] & keep, x + 8 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[w][i] = rotated ? in.cos[w][i] : 1.f;
      sn[w][i] = rotated ? in.sin[w][i] : 0.f;
    }
  }
  if (rot.interleaved) {
    rotate_pairs(cs[0], sn[0], x);
    rotate_pairs(cs[1], sn[1], x + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs[i >> 2][i & 3], s = sn[i >> 2][i & 3], lo = x[i], hi = x[8 + i];
      x[i] = lo * c - hi * s;
      x[8 + i] = hi * c + lo * s;
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t m = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
    top = top > m ? top : m;
  }
  return top;
}
// The lane's part given the row's absmax, to dst (the row's bytes) and factor.
// fma(x, s, 1.5 * 2^23 + 64) leaves w = q + 64 in its low bits, q = rne(x s):
// hi = w >> 7 and lo = (w & 127) - 64, seven bits made signed in their bytes.
template <int D>
__device__ __forceinline__ void store_query(const float (&x)[16], uint32_t top,
                                            const RotaryArgs& rot, int lane, int8_t* dst,
                                            float* factor) {
  int e[2];
  query_features<D>(rot, lane, e);
  if (top <= 0x08000000u) top = 0;   // 2^-111: 16256 / a stays finite
  const float a = __builtin_bit_cast(float, top);
  const float s = top ? 16256.0f * __builtin_amdgcn_rcpf(a) : 0.f;   // (within 2^-22 of 16256 / a)
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    v2i32 hi, lo;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = __builtin_bit_cast(uint32_t,
                                  __builtin_fmaf(x[8 * r + 4 * w + i], s, 12582912.0f + 64.f));
      const uint32_t t = (pack4(b[0], b[1], b[2], b[3]) & 0x7f7f7f7fu) ^ 0x40404040u;
      lo[w] = (int)(t | ((t & 0x40404040u) << 1));
      hi[w] = (int)pack4(b[0] >> 7, b[1] >> 7, b[2] >> 7, b[3] >> 7);
    }
    lds_store(dst + e[r], hi);
    lds_store(dst + 64 * QueryCfg<D>::kC + e[r], lo);
  }
  // An infinity leaves nothing of the row's integers to go by (inf * 0 in their
  // place): its logits are NaN or infinities of either sign, its outputs NaN.
  const float f = top < 0x7f800000u ? a * (1.0f / 16256.0f) : __builtin_nanf("");
  if (e[0] == 0) lds_store(factor, f);
}
// kPasses rows of a lane together (their reductions overlap).
template <int D, int kPasses>
__device__ __forceinline__ void row_absmax(uint32_t (&top)[kPasses]) {
#pragma unroll
  for (int d = 1; d < QueryCfg<D>::kLanes; d <<= 1)
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top[p], d, kWave);
      top[p] = top[p] > o ? top[p] : o;
    }
}
// A row's B operands: lane (row, g) holds features 64 c + 16 g .. + 15 of it.
template <int D>
__device__ __forceinline__ void read_query(const int8_t* row, int g, v4i32* hi, v4i32* lo) {
  constexpr int kC = QueryCfg<D>::kC;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    hi[c] = ld16v(row + 64 * c + 16 * g);
    lo[c] = ld16v(row + 64 * kC + 64 * c + 16 * g);
  }
}

// A wave's blocks: lane 4 i + j holds block j of its i-th group.
struct BlockList {
  int lin;            // -1 where there is no block to read
  float ks;           // key absmax / 127
  float log_a, inv_a; // of the value absmax
};

// ---- Codes through LDS. A group is staged as its four blocks, each as it lies
// in the cache, kPitch apart: 64 bytes more than a block, so that the four
// blocks a key operand touches lie in different banks. Staging is LDS-DMA, 1 KB
// an instruction, with no registers in between; the waits count its
// instructions, so each stage issues the same number of them.
template <int D>
struct Stage {
  static constexpr int kBytes = kKvBlock * D;
  static constexpr int kPitch = kBytes + 64;
  static constexpr int kLoads = (kBytes + 1023) / 1024;   // a block
  static constexpr int kGroupBytes = 4 * kPitch;
};

// Starts the copy of a block (lin in a scalar register) to dst.
template <int D>
__device__ __forceinline__ void stage_block(const int8_t* codes, int lin, int8_t* dst, int lane) {
  typedef Stage<D> S;
  const __amdgpu_buffer_rsrc_t rsrc = buffer_rsrc(codes + (int64_t)lin * S::kBytes, S::kBytes);
#pragma unroll
  for (int j = 0; j < S::kLoads; ++j) {
    if (S::kBytes % 1024 == 0 || j < S::kBytes / 1024 || lane < S::kBytes % 1024 / 16)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(dst + j * 1024), 16, lane * 16,
                                               j * 1024, 0, 0);
  }
}

// s_waitcnt with only the vector-memory counter constrained.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}
// This wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
}

// (Staged codes are read as v4i32, never as the struct uint4: a load without a
// type for alias analysis makes the compiler wait for every copy in flight.)

// A staged group's keys as the A operands of a lane (n, g): operand q of chunk
// c is token 4 q + n % 4 of block n / 4, features 64 c + 16 g .. + 15 (past D,
// where the query is zero, some other ones).
template <int D>
__device__ __forceinline__ v4i32 read_keys(const int8_t* st, int n, int g, int c, int q) {
  return *reinterpret_cast<const v4i32*>(st + (n >> 2) * Stage<D>::kPitch + (n & 3) * 16 +
                                         min(4 * c + g, D / 16 - 1) * kTile + q * 64);
}
// Its values: feature 16 d + n, the 16 tokens of block g.
template <int D>
__device__ __forceinline__ v4i32 read_values(const int8_t* st, int n, int g, int d) {
  return *reinterpret_cast<const v4i32*>(st + g * Stage<D>::kPitch + d * kTile + n * 16);
}

// One column tile's scores of a group, S^T = K Q^T as integers: element e of a
// lane is (e >> 2, e & 3) of s.
template <int D>
__device__ __forceinline__ void scores(const int8_t* st, int n, int g, const v4i32* qh,
                                       const v4i32* ql, v4i32 (&s)[4]) {
  constexpr int kC = (D + 63) / 64;
  v4i32 k[kC][4];
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) k[c][q] = read_keys<D>(st, n, g, c, q);
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = v4i32{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      s[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[c][q], qh[c], s[q], 0, 0, 0);
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = s[q] << 7;
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      s[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[c][q], ql[c], s[q], 0, 0, 0);
}

// A lane's row: its position, visible tokens and factors.
struct Row {
  int pos, lo, hi;
  float qf;      // query absmax / 16256 * scale * log2(e)
  float slope;   // * log2(e)
};

// A lane's factors of a block: weights are 2^(x f + log_a - m), and the row sum
// takes them times inv_a.
struct Scale {
  float f, log_a, inv_a;
};

// The maximum of a lane's 16 exponents. A position bias goes into x in units of
// f, its part common to the 16 into log_a. With `masked`, hidden
// tokens' x is -infinity, and a lane whose block its row does not see at all
// drops the block's factors (they may be NaN).
template <bool kAlibi>
__device__ __forceinline__ float logits(float* x, Scale* sc, const Row& row, int t0, int g,
                                        bool masked, bool here) {
  constexpr float kMinFactor = 0x1p-100f;   // (0 times -infinity would be NaN)
  sc->f *= row.qf;
  sc->f = sc->f < kMinFactor ? kMinFactor : sc->f;   // (keeps a NaN)
  const int tok0 = t0 + 16 * g;
  if (kAlibi) {
    const float step = row.slope * __builtin_amdgcn_rcpf(sc->f);
#pragma unroll
    for (int e = 1; e < 16; ++e) x[e] = __builtin_fmaf(step, (float)e, x[e]);
    sc->log_a += row.slope * (float)(tok0 - row.pos);
  }
  if (masked) {
    const int lo = row.lo - tok0, hi = row.hi - tok0;
    const bool some = here && hi > 0 && lo < 16;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = some && e >= lo && e < hi ? x[e] : -INFINITY;
    if (!some) {
      sc->f = 1.f;
      sc->log_a = sc->inv_a = 0.f;
    }
  }
  float top = fmaxf(x[0], x[1]);
#pragma unroll
  for (int e = 2; e < 16; e += 2) top = fmaxf(fmaxf(top, x[e]), x[e + 1]);
  return top * sc->f + sc->log_a;
}

// Takes a row's new maximum (over the lanes that share it) into m and l; what
// its sums over earlier tokens are to be multiplied by.
__device__ __forceinline__ float raise(float top, float* m, float* l) {
  const float next = fmaxf(*m, top - kHead);
  const float alpha = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(*m - next);
  *m = next;
  *l *= alpha;
  return alpha;
}

// The weights of four of a lane's tokens, added to sum.
__device__ __forceinline__ void weights4(const float* x, float f, float off, float* sum, float* p) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], f, -off));
  *sum += (p[0] + p[1]) + (p[2] + p[3]);
}
__device__ __forceinline__ float weight_offset(float m, const Scale& sc) {
  return (m == -INFINITY ? 0.f : m) - sc.log_a;
}

// What a row's sums over codes are multiplied by in the end (0: it saw nothing).
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.0f / (127.0f * l); }

// Four words of fp16 pairs as an MFMA operand.
__device__ __forceinline__ v8f16 as_f16(const uint32_t* w) {
  return __builtin_bit_cast(v8f16, v4i32{(int)w[0], (int)w[1], (int)w[2], (int)w[3]});
}

// The list's factors.
__device__ __forceinline__ void list_factors(float k_absmax, float v_absmax, BlockList* bl) {
  const float a = v_absmax < kMinAbsmax ? kMinAbsmax : v_absmax;   // (keeps a NaN)
  bl->ks = k_absmax / 127.0f;
  bl->log_a = __builtin_amdgcn_logf(a);
  bl->inv_a = 1.0f / a;
}

// The splits' sums of a row, weighed by their maxima, into the output of rows
// with more than one.
// Up to kFewSplits: a lane takes four features, a wave several rows. Bound by
// latency: 4096 rows of 128 features and up to 4 splits 4.9 us (a block a row 15).
constexpr int kFewSplits = 16;
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_attn_join_few(float* ws, int64_t rows,
                                                                    int splits, uint16_t* out) {
  constexpr int kLanes = D / 4, kWaveRows = kWave / kLanes;
  const int lane = threadIdx.x & 63, sub = lane / kLanes, d4 = lane % kLanes * 4;
  const int64_t row =
      ((int64_t)blockIdx.x * (kBlockThreads / kWave) + (threadIdx.x >> 6)) * kWaveRows + sub;
  if (sub >= kWaveRows || row >= rows) return;
  const Parts parts = parts_of(ws, rows, splits, D);
  const int n = min(parts.count[row], splits);
  if (n <= 1) return;
  float m[kFewSplits], top = -INFINITY, total = 0.f;
#pragma unroll
  for (int p = 0; p < kFewSplits; ++p) {
    m[p] = p < n ? parts.ml[(p * rows + row) * 2] : -INFINITY;
    top = fmaxf(top, m[p]);
  }
  const float base = top == -INFINITY ? 0.f : top;
  v4f32 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int p = 0; p < kFewSplits; ++p) {
    if (p >= n) continue;
    const float w = __builtin_amdgcn_exp2f(m[p] - base);
    total += parts.ml[(p * rows + row) * 2 + 1] * w;
    acc += ld16f(parts.o + (p * rows + row) * D + d4) * w;
  }
  acc *= inverse(total);
  *reinterpret_cast<uint2*>(out + row * D + d4) = make_uint2(f2h2(acc[0], acc[1]), f2h2(acc[2], acc[3]));
}

// More splits: one block a row. Threads take four features each, the groups of
// threads that cover a row take the splits in turn, and the groups' sums are
// added in a fixed order. 32 rows of 128 features and 64 splits: 4.7 us.
constexpr int kMaxSplits = 1024;
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_attn_join(float* ws, int64_t rows, int splits,
                                                                uint16_t* out) {
  constexpr int kLanes = D / 4, kSets = kBlockThreads / kLanes;
  __shared__ float s_w[kMaxSplits];
  __shared__ __attribute__((aligned(16))) float s_sum[kSets][D];
  __shared__ float s_red[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const Parts parts = parts_of(ws, rows, splits, D);
  const int n = min(parts.count[row], splits);
  if (n <= 1) return;
  float m[kMaxSplits / kBlockThreads], l[kMaxSplits / kBlockThreads], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kBlockThreads; ++i) {
    const int p = i * kBlockThreads + tid;
    m[i] = -INFINITY;
    l[i] = 0.f;
    if (p < n) {
      const float2 x = *reinterpret_cast<const float2*>(parts.ml + (p * rows + row) * 2);
      m[i] = x.x;
      l[i] = x.y;
    }
    top = fmaxf(top, m[i]);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
  if (lane == 0) s_red[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kBlockThreads; ++i) {
    const int p = i * kBlockThreads + tid;
    const float w = __builtin_amdgcn_exp2f(m[i] - base);
    total += l[i] * w;
    if (p < n) s_w[p] = w;
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) total += __shfl_xor(total, x, kWave);
  if (lane == 0) s_red[4 + wave] = total;
  __syncthreads();
  const int set = tid / kLanes, d4 = tid % kLanes * 4;
  if (set < kSets) {
    v4f32 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = set; p < n; p += kSets) acc += ld16f(parts.o + (p * rows + row) * D + d4) * s_w[p];
    *reinterpret_cast<v4f32*>(&s_sum[set][d4]) = acc;
  }
  __syncthreads();
  if (tid < D) {
    total = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < kSets; ++i) acc += s_sum[i][tid];
    out[row * D + tid] = f2h(acc * inverse(total));
  }
}

// The join of a launch's splits, if there are any; up to `few` by several rows a block.
template <int D>
hipError_t launch_join(float* part, int64_t rows, int splits, uint16_t* out, hipStream_t s,
                       int few = kFewSplits) {
  if (splits <= 1) return hipSuccess;
  if (splits <= few) {
    constexpr int kBlockRows = kBlockThreads / kWave * (kWave / (D / 4));
    if (rows > (int64_t)INT32_MAX * kBlockRows) return hipErrorInvalidValue;
    k_kv_attn_join_few<D><<<(uint32_t)((rows + kBlockRows - 1) / kBlockRows), kBlockThreads, 0, s>>>(
        part, rows, splits, out);
  } else {
    if (rows > INT32_MAX) return hipErrorInvalidValue;
    k_kv_attn_join<D><<<(uint32_t)rows, kBlockThreads, 0, s>>>(part, rows, splits, out);
  }
  return hipGetLastError();
}

}  // namespace

}  // namespace i8mm
