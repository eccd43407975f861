// Attention over the paged 8-bit key/value cache.
//
// Rows: the queries of one key/value head's group, row r = i * G + j for new
// token i and the j-th of the G query heads that share the head. Everything is
// computed transposed, S^T = K Q^T and O^T = V^T P^T, with the cache as the
// MFMA's A operand and 16 rows as its B operand, so that a lane keeps one row:
// lane l holds row l % 16 and, with g = l / 16, the tokens 16 g .. 16 g + 15 of
// each group of 64 (the A rows are read in that order). That is one block, so
// one key and one value absmax a lane, and the 16 weights are the B operand of
// the second product where they stand.
//
// The query is a 15-bit integer, q = (128 hi + lo) a / 16256 over its row's
// absmax a, with int8 hi and lo: two int8 MFMAs take the codes as they lie in
// the cache and sum the product exactly. That is the matrix pipe's time of one
// fp16 MFMA; it saves the conversion of the key codes and costs a shift and a
// conversion for each score. It rounds every feature by up to a / 32512: finer
// than the fp16 that the query came in for features above an eighth of a (a query
// that is not rotated would be exact in fp16), coarser for the others, and beside
// the rounding of the key codes little: over 2000 tokens of 128 features 5e-5 of
// the result against 8e-3 for normal queries, 9e-4 against 4e-2 where one feature is
// 50 times the others.
//
// Softmax in base 2. The value absmax a of a block is folded into the weight,
// P = 2^(S + log2 a - m), where m follows the running maximum of a row's S + log2 a,
// so that the products sum the value codes as they are; the row sum takes P / a, and
// O / (127 l) is the result. An a below 2^-40 counts as 2^-40, which an fp16
// result cannot tell from it. P is rounded to fp16, and the many small weights of
// a long row count like its large ones only while they round as finely: m stays
// kHead below the maximum that it was last raised to, so that P goes up to 2^15,
// the rounding is 2^-11 relative down to 2^-21 of the row's largest weight and
// 2^-32 of that below (with m at the maximum, 131000 weights of 2^-25.5 beside one
// of 1 were lost: 0.3% of the result). All sums are fp32.

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

// Rows [r, end) of a key/value head, counted on past a sequence's own, belong to
// none: their outputs are 0, and there is nothing to join. One wave.
template <int D>
__device__ __forceinline__ void zero_rows(const KvArgs& a, const AttnArgs& t, const KvSeq& sq, int h,
                                          int group, int splits, int r, int end, int lane) {
  const Parts parts = parts_of(t.part, (int64_t)a.total_tokens * t.q_heads, splits, D);
  for (; r < end; ++r) {
    const int64_t row = (int64_t)(sq.row0 + r / group) * t.q_heads + h * group + r % group;
    if (lane < D / 8) *reinterpret_cast<v4i32*>(t.out + row * D + lane * 8) = v4i32{0, 0, 0, 0};
    if (splits > 1 && lane == 0) parts.count[row] = 0;
  }
}

// Visible tokens [lo, hi) of the query at position pos.
__device__ __forceinline__ int visible_hi(const AttnArgs& t, const KvSeq& sq, int pos) {
  return pos < 0 ? 0 : t.causal ? min(pos + 1, sq.len) : sq.len;
}
__device__ __forceinline__ int visible_lo(const AttnArgs& t, int pos) {
  return t.window > 0 ? max(pos - t.window + 1, 0) : 0;
}
// Tokens that some row of new tokens i0 .. i1 sees, from a whole group on.
struct Span {
  int begin, end;
};
__device__ __forceinline__ Span row_span(const AttnArgs& t, const KvSeq& sq, int i0, int i1) {
  Span s;
  s.begin = visible_lo(t, sq.first + i0) / kGroup * kGroup;
  s.end = visible_hi(t, sq, sq.first + i1);
  return s;
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

// The blocks of 16 groups from gi0 on, `stride` apart: lane 4 i + j takes block
// j of group gi0 + i * stride; nothing at or past token `end`.
__device__ __forceinline__ void list_blocks(const KvArgs& a, int b, int h, int gi0, int stride,
                                            int end, int lane, int* lin, float* k_absmax,
                                            float* v_absmax) {
  *lin = -1;
  *k_absmax = *v_absmax = 0.f;
  const int blk = 4 * (gi0 + stride * (lane >> 2)) + (lane & 3);
  if (blk * kKvBlock < end) *lin = kv_block(a, b, h, blk);
  if (*lin >= 0) {
    *k_absmax = a.k_absmax[*lin];
    *v_absmax = a.v_absmax[*lin];
  }
}
// The list's factors.
__device__ __forceinline__ void list_factors(float k_absmax, float v_absmax, BlockList* bl) {
  const float a = v_absmax < kMinAbsmax ? kMinAbsmax : v_absmax;   // (keeps a NaN)
  bl->ks = k_absmax / 127.0f;
  bl->log_a = __builtin_amdgcn_logf(a);
  bl->inv_a = 1.0f / a;
}

// ---- Few rows: bound by the cache's bytes, each read once for all the rows of
// a key/value head. Each wave streams its own groups through its own part of
// LDS, keys and values apart: a buffer is refilled as soon as it has been read,
// so something is always in flight (a second pair of buffers changed nothing). The
// four waves of a block join through LDS, the blocks of a row tile through the
// workspace and the kernels below. The weights go to the second product in two
// parts of fp16: there is time for it. One token over each of 64 sequences of up to
// 8192, 64 heads on 8 of 128 features (595 MB): 117 us, 5.1 TB/s, and 5 us to join;
// over one of 131071, 32 heads on 8 (268 MB): 51 us, 5.3 TB/s, and 5 us. A large
// copy moves 5.2 TB/s on the same card.
template <int D, bool kAlibi>
__global__ __launch_bounds__(kBlockThreads, D <= 128 ? 2 : 1) void k_kv_attn_rows(KvArgs a, RotaryArgs rot,
                                                                AttnArgs t, int group, int tiles,
                                                                int splits, int chunk) {
  constexpr int kC = (D + 63) / 64, kT = D / 16, kLd = D + 4;
  typedef Stage<D> S;
  constexpr int kAhead = 4 * S::kLoads;   // loads younger than the awaited: the other buffer's
  constexpr int kJoinBytes = (4 * kRows * kLd + 8 * kRows) * 4;
  constexpr int kStageBytes = 4 * 2 * S::kGroupBytes;
  typedef QueryCfg<D> Q;
  __shared__ __attribute__((aligned(1024)))
  int8_t lds[(kStageBytes > kJoinBytes ? kStageBytes : kJoinBytes) + kRows * (Q::kRowBytes + 4)];
  int8_t* const lds_q = lds + (sizeof(lds) - kRows * (Q::kRowBytes + 4));
  float* const s_qf = reinterpret_cast<float*>(lds_q + kRows * Q::kRowBytes);
  float(*s_o)[kRows][kLd] = reinterpret_cast<float(*)[kRows][kLd]>(lds);
  float(*s_m)[kRows] = reinterpret_cast<float(*)[kRows]>(lds + 4 * kRows * kLd * 4);
  float(*s_l)[kRows] = s_m + 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int h = blockIdx.x / tiles, b = blockIdx.y;
  const int r_first = (blockIdx.x % tiles) * kRows;
  const KvSeq sq = kv_seq(a, b);
  const int rows = sq.n * group;
  if (sq.row0 + sq.n < sq.stop) {
    // the rows after the sequence's that belong to none, over all its blocks: their
    // outputs are 0, and there is nothing to join
    const int64_t first = (int64_t)(sq.row0 + sq.n) * t.q_heads;
    const int64_t past = (int64_t)sq.stop * t.q_heads;
    const int64_t threads = (int64_t)gridDim.x * gridDim.z * kBlockThreads;
    const int64_t at = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * kBlockThreads + threadIdx.x;
    for (int64_t i = first * (D / 8) + at; i < past * (D / 8); i += threads)
      *reinterpret_cast<v4i32*>(t.out + i * 8) = v4i32{0, 0, 0, 0};
    if (splits > 1) {
      const Parts parts = parts_of(t.part, (int64_t)a.total_tokens * t.q_heads, splits, D);
      for (int64_t i = first + at; i < past; i += threads) parts.count[i] = 0;
    }
  }
  if (r_first >= rows) return;
  const int r_last = min(r_first + kRows, rows) - 1;
  const Span span = row_span(t, sq, r_first / group, r_last / group);
  // Whole chunks first, then what is left of each span together, since what starts
  // last should be short: in the slab that the longest sequence's rest falls into
  // (the last is for spans that begin inside a group). Against a sequence's chunks
  // one after the other, 16 ragged sequences of 32 heads 65.1 us and 67.6, 64 of
  // grouped heads 122.2 and 123.6; with 256 features 64 sequences 128 and 123.
  const int whole = min((span.end - span.begin) / chunk, splits - 1), z = blockIdx.z;
  if (z >= whole && z != max(whole, splits - 2)) return;
  const int split = min(z, whole);
  const int begin = span.begin + split * chunk;
  // an empty span still has its outputs written, by split 0
  if (split > 0 && begin >= span.end) return;
  const int end = min(begin + chunk, span.end);
  const bool only = span.end - span.begin <= chunk;

  const int r = min(r_first + n, r_last);
  const bool live = r_first + n <= r_last;
  const int i_row = r / group, head = h * group + r % group;
  Row row;
  row.pos = sq.first + i_row;
  // the waves share the queries' preparation
  constexpr int kPasses = (kRows + 4 * Q::kPassRows - 1) / (4 * Q::kPassRows);
  QueryLoads q_in[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = min(r_first + (4 * p + wave) * Q::kPassRows + lane / Q::kLanes, r_last);
    load_query<D>(t.q + (int64_t)(sq.row0 + rr / group) * t.q_ts +
                      (int64_t)(h * group + rr % group) * t.q_hs,
                  max(sq.first + rr / group, 0), rot, t.q, lane, q_in[p]);
  }
  v4i32 qh[kC], ql[kC];
  row.lo = visible_lo(t, row.pos);
  row.hi = live ? visible_hi(t, sq, row.pos) : 0;
  row.slope = kAlibi ? t.slopes[head] * 1.44269504088896340736f : 0.f;
  // groups inside [all_lo, all_hi) are visible to every row
  const int all_lo = visible_lo(t, sq.first + r_last / group);
  const int all_hi = visible_hi(t, sq, sq.first + r_first / group);

  v4f32 o[kT];
#pragma unroll
  for (int d = 0; d < kT; ++d) o[d] = v4f32{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  const int gi_end = (end + kGroup - 1) / kGroup;
  const int gi_first = begin / kGroup + wave;
  int8_t* const st_k = lds + wave * (2 * S::kGroupBytes);
  int8_t* const st_v = st_k + S::kGroupBytes;
  BlockList bl;
  float k_absmax, v_absmax;
  // absent blocks are masked; block 0 is read in their place
  auto load = [&](int i, const int8_t* codes, int8_t* dst) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      stage_block<D>(codes, max(__builtin_amdgcn_readlane(bl.lin, 4 * i + j), 0),
                     dst + j * S::kPitch, lane);
  };
  // the list of 16 groups from gi0 on, and the first group's copies
  auto start = [&](int gi0) __attribute__((always_inline)) {
    list_blocks(a, b, h, gi0, 4, end, lane, &bl.lin, &k_absmax, &v_absmax);
    load(0, a.k_codes, st_k);
    load(0, a.v_codes, st_v);
  };
  if (gi_first < gi_end) start(gi_first);
  // (the codes are on their way meanwhile)
  float x_in[kPasses][16];
  uint32_t x_top[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = r_first + (4 * p + wave) * Q::kPassRows + lane / Q::kLanes;
    x_top[p] = rotate_query<D>(q_in[p], r <= r_last && sq.first + r / group >= 0, rot, lane, x_in[p]);
  }
  row_absmax<D>(x_top);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = (4 * p + wave) * Q::kPassRows + lane / Q::kLanes;
    if (rr < kRows) store_query<D>(x_in[p], x_top[p], rot, lane, lds_q + rr * Q::kRowBytes, s_qf + rr);
  }
  lds_only_barrier();
  read_query<D>(lds_q + n * Q::kRowBytes, g, qh, ql);
  row.qf = s_qf[n] * t.scale_log2;

  for (int gi0 = gi_first; gi0 < gi_end; gi0 += 64) {
    if (gi0 != gi_first) {
      wait_lds_reads();   // of the list before
      start(gi0);
    }
    const uint64_t present = __ballot(bl.lin >= 0);
    const int count = min(16, (gi_end - gi0 + 3) / 4);
    list_factors(k_absmax, v_absmax, &bl);
    for (int i = 0; i < count; ++i) {
      const uint32_t have = (uint32_t)(present >> (4 * i)) & 15u;
      const int t0 = (gi0 + 4 * i) * kGroup;
      v4i32 s[4];
      float x[16], p[16];
      if (i + 1 < count) wait_loads<kAhead>(); else wait_loads<0>();
      scores<D>(st_k, n, g, qh, ql, s);
      if (i + 1 < count) {
        wait_lds_reads();
        load(i + 1, a.k_codes, st_k);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = (float)s[e >> 2][e & 3];
      Scale sc = {__shfl(bl.ks, 4 * i + g, kWave), __shfl(bl.log_a, 4 * i + g, kWave),
                  __shfl(bl.inv_a, 4 * i + g, kWave)};
      const float top = max_over_groups<4>(
          logits<kAlibi>(x, &sc, row, t0, g, t0 < all_lo || t0 + kGroup > all_hi || have != 15u,
                         (have >> g) & 1u));
      if (__any(top > m + (kHead + kLazy))) {
        const float alpha = raise(top, &m, &l);
#pragma unroll
        for (int d = 0; d < kT; ++d) o[d] *= alpha;
      }
      const float off = weight_offset(m, sc);
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) weights4(x + 4 * q, sc.f, off, &sum, p + 4 * q);
      l += sum * sc.inv_a;
      uint32_t ph[8], pl[8];   // the weights in two parts of 11 bits
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ph[e] = f2h2(p[2 * e], p[2 * e + 1]);
        pl[e] = f2h2(p[2 * e] - h2f(ph[e] & 0xffffu), p[2 * e + 1] - h2f(ph[e] >> 16));
      }
      const v8f16 p0h = as_f16(ph), p1h = as_f16(ph + 4), p0l = as_f16(pl), p1l = as_f16(pl + 4);
      if (i + 1 < count) wait_loads<kAhead>(); else wait_loads<0>();
#pragma unroll
      for (int d = 0; d < kT; ++d) {
        v8f16 v0, v1;
        codes_to_f16(read_values<D>(st_v, n, g, d), &v0, &v1);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0l, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1l, o[d], 0, 0, 0);
      }
      if (i + 1 < count) {
        wait_lds_reads();
        load(i + 1, a.v_codes, st_v);
      }
    }
  }

  // join the four waves
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  __syncthreads();   // every wave is done with the staged groups
#pragma unroll
  for (int d = 0; d < kT; ++d) *reinterpret_cast<v4f32*>(&s_o[wave][n][16 * d + 4 * g]) = o[d];
  if (g == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
  }
  __syncthreads();
  const Parts parts = parts_of(t.part, (int64_t)a.total_tokens * t.q_heads, splits, D);
  for (int x = threadIdx.x; x < kRows * (D / 4); x += kBlockThreads) {
    const int row = x / (D / 4), d4 = x % (D / 4) * 4;
    if (r_first + row > r_last) continue;
    float top = s_m[0][row];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, s_m[w][row]);
    const float base = top == -INFINITY ? 0.f : top;
    v4f32 acc = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float e = __builtin_amdgcn_exp2f(s_m[w][row] - base);
      total += s_l[w][row] * e;
      acc += *reinterpret_cast<const v4f32*>(&s_o[w][row][d4]) * e;
    }
    const int rr = r_first + row;
    const int64_t out_row = (int64_t)(sq.row0 + rr / group) * t.q_heads + h * group + rr % group;
    if (only) {
      const float inv = inverse(total);
      *reinterpret_cast<uint2*>(t.out + out_row * D + d4) =
          make_uint2(f2h2(acc[0] * inv, acc[1] * inv), f2h2(acc[2] * inv, acc[3] * inv));
    } else {
      const int64_t part = split * parts.rows + out_row;
      *reinterpret_cast<v4f32*>(parts.o + part * D + d4) = acc;
      if (d4 == 0) {
        parts.ml[part * 2] = top;
        parts.ml[part * 2 + 1] = total;
      }
    }
    if (splits > 1 && split == 0 && d4 == 0)
      parts.count[out_row] = (span.end - span.begin + chunk - 1) / chunk;
  }
}

// ---- Many rows: the waves of a block share each group, a wave takes kR rows: 32
// by MFMAs of 32 x 32 (half the instructions of 16 x 16, which keep the vector
// pipe from issuing; the two lanes of a row hold two blocks of a group each) or 16
// as above, where there is not work enough (see the plan) and for D = 256, whose
// sums of 32 rows would not leave room. Keys are copied to LDS as they are, into
// the next of three buffers. Values are turned into fp16 once for the block
// (converted by every wave for itself they were a third of its vector
// instructions): each wave loads its share of a group one step ahead and stores it
// as operands, of which LDS holds this group's and the next's.
//
// 4096 tokens of 96 heads of 128 (412 GFLOP): 520 to 550 us, 0.75 to 0.79 PFLOP/s (a
// large fp16 product: 1.2). The vector pipe is busy for 0.62 of the cycles at 2.05
// GHz (about 270 instructions beside 32 MFMAs for a group of 64 tokens, 32 rows and
// 128 features: exponentials, conversions, the joining of the two parts of the
// scores), the matrix pipe for 0.38. Neither is full: they take turns more than they
// overlap, with two waves a SIMD and a barrier every 64 tokens. A step of prompt
// chunks over prefixes of up to 8191 tokens, 32 heads on 8 of 64 (90 GFLOP): 178 us,
// 0.63 and 0.20 of the cycles. What else it costs a block is its start, about 12 us for
// the queries.
template <int D, int kR>
struct TileCfg {
  static constexpr int kLaneGroups = kWave / kR;        // lanes of a row
  static constexpr int kBlocks = 4 / kLaneGroups;       // blocks of a group a lane holds
  static constexpr int kTiles = kGroup / kR;            // score tiles of a group
  static constexpr int kValues = 16 * kBlocks / kTiles; // of a lane, of a score tile
  static constexpr int kChunk = 16 * kLaneGroups;       // features of an int8 MFMA
  static constexpr int kC = (D + kChunk - 1) / kChunk;
  static constexpr int kO = (D + kR - 1) / kR;          // output tiles of kR features
  static constexpr int kWaves = D <= 128 ? 4 : 8;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kBlockRows = kWaves * kR;
  static constexpr int kKeyBuffers = 3;
  static constexpr int kKeyLoads = 4 * Stage<D>::kLoads / kWaves;   // a wave's, of a group
  static constexpr int kValueTiles = (D / 16 + kWaves - 1) / kWaves;
  // (room for every wave's tiles: those past D / 16 are copies nobody reads)
  static constexpr int kValueBytes = kWaves * kValueTiles * 2048;
  static constexpr int kValues0 = kKeyBuffers * Stage<D>::kGroupBytes;
  static constexpr int kFactors0 = kValues0 + 2 * kValueBytes;
  static constexpr int kQueryFactors0 = kFactors0 + kWaves * kWave * 16;
  static constexpr int kLds = kQueryFactors0 + kBlockRows * 4;
  // (the queries stand where values will)
  static_assert(kBlockRows * QueryCfg<D>::kRowBytes <= 2 * kValueBytes, "room for the queries");
  static_assert(kO * kR <= kWaves * kValueTiles * 16, "operands of every output tile");
};

__device__ __forceinline__ v16i32 mfma_i8(v4i32 a, v4i32 b, v16i32 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4i32 mfma_i8(v4i32 a, v4i32 b, v4i32 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f32 mfma_f16(v8f16 a, v8f16 b, v16f32 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f32 mfma_f16(v8f16 a, v8f16 b, v4f32 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The keys of score tile q as an operand. Its rows are taken such that a lane's
// values over the tiles are the tokens of its first block in order, then those
// of its second.
template <int D, int kR>
__device__ __forceinline__ void read_key_tile(const int8_t* st, int n, int g, int q,
                                              v4i32 (&k)[TileCfg<D, kR>::kC]) {
  typedef TileCfg<D, kR> Cfg;
  const int8_t* p = st + (kR == 32
                              ? (2 * q + ((n >> 2) & 1)) * Stage<D>::kPitch + 64 * (n >> 3)
                              : (n >> 2) * Stage<D>::kPitch + 64 * q) + 16 * (n & 3);
#pragma unroll
  for (int c = 0; c < Cfg::kC; ++c) {
    // (a lane past the last feature meets zeros of the query)
    const int tile = Cfg::kLaneGroups * c + g;
    k[c] = ld16v(p + (D % Cfg::kChunk == 0 ? tile : min(tile, D / 16 - 1)) * kTile);
  }
}

// What a block does. Heads come first in the block index: blocks go to the 8
// XCDs in turn, so with a multiple of 8 heads a head's blocks share one L2. A
// head's blocks take the longest sequence first, of each the last tiles first
// (causal rows see more tokens the later they are): what starts last should be
// short. Blocks without work come last: among the others, they upset the turns
// in which blocks go to compute units (a step of mixed prompt chunks took
// twice as long). A wave's lanes hold a sequence each, up to 64 of them.
struct Place {
  int b, tile, split;   // b < 0: nothing to do
};

// Tiles of a sequence and of the rows after it that belong to none.
template <int kTileRows>
__device__ __forceinline__ int tiles_of(const KvSeq& sq, int group) {
  return ((sq.stop - sq.row0) * group + kTileRows - 1) / kTileRows;
}

// More than 64 sequences are taken in order, split by split. Tiles of packed rows:
// sequence b's begin at slot floor(cu_tokens[b] group / kTileRows) + b, so each
// has room for its own and at most one is empty, and the sequence of a slot is
// found by a search of 64 probes at once.
template <int kTileRows>
__host__ __device__ __forceinline__ int64_t first_slot(int64_t row, int group, int b) {
  return row * group / kTileRows + b;
}
template <int kTileRows>
__device__ __forceinline__ Place place_among_many(const KvArgs& a, int job, int group, int lane) {
  const int slots = (int)first_slot<kTileRows>(a.total_tokens, group, a.num_seqs);
  const int split = job / slots, slot = job - split * slots;
  int b = 0;   // of [b, b + size), the last whose tiles begin at `slot` or before
  for (int size = a.num_seqs; size > 0;) {
    const int step = (size + kWave - 1) / kWave, ahead = lane * step;
    bool before = false;
    if (ahead < size) {
      const int at = b + ahead;
      const int row = a.cu_tokens ? min(max(a.cu_tokens[at], 0), a.total_tokens) : at;
      before = first_slot<kTileRows>(row, group, at) <= slot;
    }
    const uint64_t some = __ballot(before);
    if (!some) return Place{-1, 0, 0};
    const int skip = (63 - __builtin_clzll(some)) * step;
    b += skip;
    size = step > 1 ? min(step, size - skip) : 0;
  }
  const KvSeq sq = kv_seq(a, b);
  const int tile = slot - (int)first_slot<kTileRows>(sq.row0, group, b);
  const int own = tiles_of<kTileRows>(sq, group);
  return tile < own ? Place{b, own - 1 - tile, split} : Place{-1, 0, 0};
}

template <int kTileRows>
__device__ __forceinline__ Place place_of(const KvArgs& a, const AttnArgs& t, int job, int group,
                                          int chunk, int lane) {
  // (marked as rare, or a step of chunks takes 2% longer)
  if (__builtin_expect(a.num_seqs > kWave, 0)) return place_among_many<kTileRows>(a, job, group, lane);
  int my_tiles = 0, my_splits = 0, len = -1;
  if (lane < a.num_seqs) {
    const KvSeq sq = kv_seq(a, lane);
    len = sq.len;
    my_tiles = tiles_of<kTileRows>(sq, group);
    int seen = t.window > 0 ? min(len, t.window + sq.n) + kGroup : len;
    my_splits = max((seen + chunk - 1) / chunk, 1);
  }
  const int jobs = my_tiles * my_splits;
  int start = 0;
  for (int k = 0; k < a.num_seqs; ++k) {
    const int other = __builtin_amdgcn_readlane(len, k), n = __builtin_amdgcn_readlane(jobs, k);
    start += other > len || (other == len && k < lane) ? n : 0;
  }
  const uint64_t mine = __ballot(job >= start && job < start + jobs);
  if (!mine) return Place{-1, 0, 0};
  const int b = __builtin_ctzll(mine);
  const int in = job - __builtin_amdgcn_readlane(start, b);
  const int s = __builtin_amdgcn_readlane(my_splits, b);
  return Place{b, __builtin_amdgcn_readlane(my_tiles, b) - 1 - in / s, in % s};
}

template <int D, int kR, bool kAlibi>
__global__ __launch_bounds__((TileCfg<D, kR>::kThreads), 2) void k_kv_attn_tile(
    KvArgs a, RotaryArgs rot, AttnArgs t, int group, int splits, int chunk) {
  typedef Stage<D> S;
  typedef TileCfg<D, kR> Cfg;
  constexpr int kC = Cfg::kC, kT = Cfg::kBlocks, kO = Cfg::kO;
  constexpr int kTiles = Cfg::kTiles, kValues = Cfg::kValues;
  // loads of a wave younger than the keys it waits for: the next group's keys
  // and its own values of that group
  constexpr int kAhead = Cfg::kKeyLoads + Cfg::kValueTiles;
  __shared__ __attribute__((aligned(1024))) int8_t lds[Cfg::kLds];
  int8_t* const lds_v = lds + Cfg::kValues0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane % kR, g = lane / kR;            // row, lane group
  const int n16 = lane & 15, g16 = lane >> 4;
  const int h = blockIdx.x % a.kv_heads;
  const Place at =
      place_of<Cfg::kBlockRows>(a, t, blockIdx.x / a.kv_heads, group, chunk, lane);
  const int b = at.b;
  if (b < 0) return;
  const KvSeq sq = kv_seq(a, b);
  const int rows = sq.n * group;
  const int blk_first = at.tile * Cfg::kBlockRows;
  const bool zeros = blk_first + Cfg::kBlockRows > rows && sq.row0 + sq.n < sq.stop && at.split == 0;
  if (__builtin_expect(zeros, 0)) {
    const int r = blk_first + wave * kR, all = (sq.stop - sq.row0) * group;
    zero_rows<D>(a, t, sq, h, group, splits, max(r, rows), min(r + kR, all), lane);
  }
  if (blk_first >= rows) return;
  const int blk_last = min(blk_first + Cfg::kBlockRows, rows) - 1;
  const Span span = row_span(t, sq, blk_first / group, blk_last / group);
  const int begin = span.begin + at.split * chunk;
  if (at.split > 0 && begin >= span.end) return;
  const int end = min(begin + chunk, span.end);
  const bool only = span.end - span.begin <= chunk;

  // the wave's rows (none: it stages, and computes nothing)
  const int w_first = blk_first + wave * kR;
  const int w_last = min(w_first + kR, rows) - 1;
  const int i_first = min(w_first, rows - 1) / group, i_last = max(w_last, 0) / group;
  const int all_lo = visible_lo(t, sq.first + i_last);
  const int all_hi = visible_hi(t, sq, sq.first + i_first);
  const bool works = w_first < rows;

  int lin, lin_next = -1;
  float ka, va, ka_next = 0.f, va_next = 0.f;
  const int gi_begin = begin / kGroup, gi_end = (end + kGroup - 1) / kGroup;
  list_blocks(a, b, h, gi_begin, 1, end, lane, &lin, &ka, &va);
  // What follows takes group gi as the i-th (up to 31st) of the current and
  // the next list. Absent blocks are masked; block 0 is read in their place, and
  // past the last group too (so that each step issues the same loads).
  auto stage_keys = [&](int gi, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int jj = 0; jj < Cfg::kKeyLoads; ++jj) {
      const int blk = (wave * Cfg::kKeyLoads + jj) / S::kLoads, j = (wave * Cfg::kKeyLoads + jj) % S::kLoads;
      const int x = i < 16 ? __builtin_amdgcn_readlane(lin, (4 * i + blk) & 63)
                           : __builtin_amdgcn_readlane(lin_next, (4 * i + blk) & 63);
      const __amdgpu_buffer_rsrc_t rsrc =
          buffer_rsrc(a.k_codes + (int64_t)max(x, 0) * S::kBytes, S::kBytes);
      int8_t* dst = lds + gi % Cfg::kKeyBuffers * S::kGroupBytes + blk * S::kPitch + j * 1024;
      if (S::kBytes % 1024 == 0 || j < S::kBytes / 1024 || lane < S::kBytes % 1024 / 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)dst, 16, lane * 16, j * 1024, 0, 0);
    }
  };
  v4i32 vr[Cfg::kValueTiles];   // the wave's tiles of a group: wave, wave + kWaves, ..
  auto load_values = [&](int i) __attribute__((always_inline)) {
    const int x = __shfl(i < 16 ? lin : lin_next, (4 * i + g16) & 63, kWave);
    const int8_t* p = a.v_codes + (int64_t)max(x, 0) * S::kBytes + n16 * 16;
#pragma unroll
    for (int j = 0; j < Cfg::kValueTiles; ++j)
      vr[j] = ld16v(p + min(wave + j * Cfg::kWaves, D / 16 - 1) * kTile);
  };
  // Features 16 d + n16, block g16, to the operands of the second product: 1 KB for
  // each output tile, block of a lane and half of it, the lane's 8 tokens in 16
  // bytes.
  auto store_value_tile = [&](int gi, int j) __attribute__((always_inline)) {
    const int d = wave + j * Cfg::kWaves;
    int8_t* dst = lds_v + (gi & 1) * Cfg::kValueBytes;
    if constexpr (kR == 32)
      dst += (d >> 1) * 4096 + (g16 >> 1) * 2048 + (16 * (d & 1) + n16 + 32 * (g16 & 1)) * 16;
    else
      dst += d * 2048 + lane * 16;
    v8f16 v0, v1;
    codes_to_f16(vr[j], &v0, &v1);
    lds_store(dst, __builtin_bit_cast(v4i32, v0));
    lds_store(dst + 1024, __builtin_bit_cast(v4i32, v1));
  };
  auto store_values = [&](int gi) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < Cfg::kValueTiles; ++j) store_value_tile(gi, j);
  };
  if (gi_begin < gi_end) {
    load_values(0);
    stage_keys(gi_begin, 0);
    stage_keys(gi_begin + 1, 1);
    stage_keys(gi_begin + 2, 2);
  }
  typedef QueryCfg<D> Q;
  constexpr int kPasses = kR / Q::kPassRows;
  int8_t* const lds_q = lds_v + wave * (kR * Q::kRowBytes);
  float* const s_qf = reinterpret_cast<float*>(lds + Cfg::kQueryFactors0) + wave * kR;
  QueryLoads q_in[kPasses];
  // token and head of the lane's row, pass by pass without a division each
  const int tok_last = (rows - 1) / group, j_last = rows - 1 - tok_last * group;
  const int tok_step = Q::kPassRows / group, j_step = Q::kPassRows - tok_step * group;
  int tok = (w_first + lane / Q::kLanes) / group, j = w_first + lane / Q::kLanes - tok * group;
  uint32_t sees = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const bool live = w_first + p * Q::kPassRows + lane / Q::kLanes < rows;
    const int tok_p = live ? tok : tok_last, j_p = live ? j : j_last, pos = sq.first + tok_p;
    load_query<D>(t.q + (int64_t)(sq.row0 + tok_p) * t.q_ts + (int64_t)(h * group + j_p) * t.q_hs,
                  max(pos, 0), rot, t.q, lane, q_in[p]);
    sees |= (live && pos >= 0 ? 1u : 0u) << p;
    tok += tok_step;
    j += j_step;
    if (j >= group) {
      j -= group;
      ++tok;
    }
  }
  float x_in[kPasses][16];
  uint32_t x_top[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
    x_top[p] = rotate_query<D>(q_in[p], (sees >> p) & 1u, rot, lane, x_in[p]);
  row_absmax<D>(x_top);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = p * Q::kPassRows + lane / Q::kLanes;
    store_query<D>(x_in[p], x_top[p], rot, lane, lds_q + rr * Q::kRowBytes, s_qf + rr);
  }
  Row row;
  v4i32 qh[kC], ql[kC];
  const int r = min(w_first + n, rows - 1), i_row = r / group, head = h * group + r % group;
  const bool live = w_first + n < rows;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    qh[c] = ld16v(lds_q + n * Q::kRowBytes + Cfg::kChunk * c + 16 * g);
    ql[c] = ld16v(lds_q + n * Q::kRowBytes + Q::kRowBytes / 2 + Cfg::kChunk * c + 16 * g);
  }
  row.qf = s_qf[n] * t.scale_log2;
  row.pos = sq.first + i_row;
  row.lo = visible_lo(t, row.pos);
  row.hi = live ? visible_hi(t, sq, row.pos) : 0;
  row.slope = kAlibi ? t.slopes[head] * 1.44269504088896340736f : 0.f;
  lds_only_barrier();   // every wave has its queries
  if (gi_begin < gi_end) {
    store_values(gi_begin);
    load_values(1);
  }
  typedef typename std::conditional<kR == 32, v16f32, v4f32>::type OTile;
  OTile o[kO];
#pragma unroll
  for (int d = 0; d < kO; ++d) o[d] = OTile{};
  float m = -INFINITY, l = 0.f;

  // the list's factors, a copy for each wave: lane 4 i + j, block j of group i
  v4f32* const s_factors = reinterpret_cast<v4f32*>(lds + Cfg::kFactors0) + wave * kWave;
  uint64_t present;
  auto take_list = [&]() __attribute__((always_inline)) {
    BlockList bl;
    present = __ballot(lin >= 0);
    list_factors(ka, va, &bl);
    lds_store(reinterpret_cast<int8_t*>(s_factors + lane),
              __builtin_bit_cast(v4i32, v4f32{bl.ks, bl.log_a, bl.inv_a, 0.f}));
  };
  take_list();
  float x[16 * kT], top = -INFINITY;
  Scale sc[kT];
  // factors of the list's i-th group
  auto factors = [&](int i, v4f32 (&f)[kT]) __attribute__((always_inline)) {
#pragma unroll
    for (int T = 0; T < kT; ++T) f[T] = s_factors[4 * i + Cfg::kLaneGroups * T + g];
  };
  // the maximum of group gi, the i-th of the list
  auto maximum = [&](int gi, int i, const v4f32 (&f)[kT]) __attribute__((always_inline)) {
    const int t0 = gi * kGroup;
    const uint32_t have = (uint32_t)(present >> (4 * i)) & 15u;
    const bool masked = t0 < all_lo || t0 + kGroup > all_hi || have != 15u;
    top = -INFINITY;
#pragma unroll
    for (int T = 0; T < kT; ++T) {
      const int blk = Cfg::kLaneGroups * T + g;
      sc[T] = Scale{f[T][0], f[T][1], f[T][2]};
      top = fmaxf(top, logits<kAlibi>(x + 16 * T, &sc[T], row, t0, blk, masked, (have >> blk) & 1u));
    }
    top = max_over_groups<Cfg::kLaneGroups>(top);
  };
  typedef typename std::conditional<kR == 32, v16i32, v4i32>::type STile;
  // a score tile; between its two halves, `middle`
  auto products = [&](const v4i32 (&k)[kC], auto middle) __attribute__((always_inline)) {
    STile acc = {};
#pragma unroll
    for (int c = 0; c < kC; ++c) acc = mfma_i8(k[c], qh[c], acc);
    middle();
    acc = acc << 7;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc = mfma_i8(k[c], ql[c], acc);
    return acc;
  };
  STile s[kTiles];
  if (gi_begin < gi_end) {
    wait_loads<kAhead>();
    lds_only_barrier();
    if (works) {
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        v4i32 k[kC];
        read_key_tile<D, kR>(lds + gi_begin % Cfg::kKeyBuffers * S::kGroupBytes, n, g, q, k);
        s[q] = products(k, [] {});
#pragma unroll
        for (int e = 0; e < kValues; ++e) x[q * kValues + e] = (float)s[q][e];
      }
      v4f32 f[kT];
      factors(0, f);
      maximum(gi_begin, 0, f);
    }
  }

  // Step gi: the products of group gi + 1 beside the weights of group gi, then
  // the values of group gi beside the conversion of those products: the matrix
  // pipe works on one group while the vector pipe works on the other.
  for (int gi = gi_begin; gi < gi_end; ++gi) {
    const int i = (gi - gi_begin) & 15;
    if (i == 0 && gi + 16 < gi_end)
      list_blocks(a, b, h, gi + 16, 1, end, lane, &lin_next, &ka_next, &va_next);
    wait_loads<kAhead>();
    // the keys of gi + 1 and the values of gi are in LDS; every wave is done
    // with the keys of gi and the values of gi - 1
    lds_only_barrier();
    stage_keys(gi + 3, i + 3);
    v4f32 next[kT];
    if (works) {
      if (__any(top > m + (kHead + kLazy))) {
        const float alpha = raise(top, &m, &l);
#pragma unroll
        for (int d = 0; d < kO; ++d) o[d] *= alpha;
      }
      // (the keys past the last group are what the buffer holds)
      const int8_t* st_k = lds + (gi + 1) % Cfg::kKeyBuffers * S::kGroupBytes;
      const int8_t* st_v = lds_v + (gi & 1) * Cfg::kValueBytes + lane * 16;
      uint32_t pw[8 * kT];
      v4i32 k[kTiles][kC], v[kO * kT][2];
      // LDS reads run kValueAhead pairs of operands ahead
      constexpr int kValueAhead = 1;
      auto read_v = [&](int i) __attribute__((always_inline)) {
        v[i][0] = ld16v(st_v + i * 2048);
        v[i][1] = ld16v(st_v + i * 2048 + 1024);
      };
      read_key_tile<D, kR>(st_k, n, g, 0, k[0]);
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        if (q + 1 == kTiles)
#pragma unroll
          for (int i = 0; i < kValueAhead; ++i) read_v(i);
        s[q] = products(k[q], [&]() __attribute__((always_inline)) {
          // weights of group gi (the row sum takes them unrounded: those of a block
          // of far smaller values vanish in fp16)
          const Scale& of = sc[q * kValues / 16];
          const float off = weight_offset(m, of);
          float sum = 0.f;
#pragma unroll
          for (int w = q * kValues / 2; w < (q + 1) * kValues / 2; ++w) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * w], of.f, -off));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * w + 1], of.f, -off));
            sum += p0 + p1;
            pw[w] = f2h2(p0, p1);
          }
          l += sum * of.inv_a;
        });
        if (q + 1 < kTiles) read_key_tile<D, kR>(st_k, n, g, q + 1, k[q + 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      factors((i + 1) & 15, next);
#pragma unroll
      for (int dT = 0; dT < kO * kT; ++dT) {
        const int d = dT / kT, T = dT % kT;
        if (dT + kValueAhead < kO * kT) read_v(dT + kValueAhead);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          o[d] = mfma_f16(__builtin_bit_cast(v8f16, v[dT][u]), as_f16(pw + 8 * T + 4 * u), o[d]);
#pragma unroll
        for (int e = 0; e < 16 * kT; ++e)
          if (e * kO / 16 == dT) x[e] = (float)s[e / kValues][e % kValues];
#pragma unroll
        for (int j = 0; j < Cfg::kValueTiles; ++j)
          if (dT == j * (kO * kT / Cfg::kValueTiles)) store_value_tile(gi + 1, j);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      store_values(gi + 1);
    }
    load_values(i + 2);
    if (i == 15) {   // the next list, if any
      lin = lin_next;
      ka = ka_next;
      va = va_next;
      take_list();
      factors(0, next);
    }
    if (works && gi + 1 < gi_end) maximum(gi + 1, (i + 1) & 15, next);
  }
  wait_loads<0>();   // nothing may land in LDS after the block has ended

  const Parts parts = parts_of(t.part, (int64_t)a.total_tokens * t.q_heads, splits, D);
  if constexpr (Cfg::kLaneGroups == 4) l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (!live) return;
  const int64_t out_row = (int64_t)(sq.row0 + i_row) * t.q_heads + head;
  // a lane's sums: of each output tile, runs of four features
  constexpr int kRuns = kR == 32 ? 4 : 1;
  const float inv = inverse(l);
  const int64_t part = at.split * parts.rows + out_row;
#pragma unroll
  for (int d = 0; d < kO; ++d)
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      const int e0 = d * kR + 8 * k + 4 * g;
      if (D % kR != 0 && e0 >= D) continue;
      const v4f32 y = {o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]};
      if (only)
        *reinterpret_cast<uint2*>(t.out + out_row * D + e0) =
            make_uint2(f2h2(y[0] * inv, y[1] * inv), f2h2(y[2] * inv, y[3] * inv));
      else
        *reinterpret_cast<v4f32*>(parts.o + part * D + e0) = y;
    }
  if (g == 0 && !only) {
    parts.ml[part * 2] = m;
    parts.ml[part * 2 + 1] = l;
  }
  if (g == 0 && splits > 1 && at.split == 0)
    parts.count[out_row] = (span.end - span.begin + chunk - 1) / chunk;
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

struct Plan {
  bool shared, wide;   // the kernel for many rows; its waves of 32 rows
  int group, tile_rows, tiles, splits, chunk;
};

// Tiles of all sequences together, at most.
int64_t most_tiles(const KvArgs& a, const Plan& p) {
  return std::min((int64_t)p.tiles * a.num_seqs,
                  (int64_t)a.total_tokens * p.group / p.tile_rows + a.num_seqs);
}

// Which kernel: up to 48 rows the one for few rows, each 16 of them another block
// (8 sequences of up to 8191 tokens, 8 heads: 48 rows of 64 features 26 us against
// 31, of 80 features 36 against 40, of 128 alike; 64 rows 34 against 28 and 46
// against 36 of 64 and 128); of 256 features up to 32 (48 rows 82 us against 86, but
// 50 against 30 where one sequence is alone).
// Waves of 32 rows where there is work for them, measured by the tokens that a
// resident block of 128 rows would take; the fewer features, the less a wave gains
// from more rows (80 fill three output tiles of 32 to five sixths). Prompts of
// 1024 to 4096 tokens, against waves of 16 rows, with that share: 128 features
// (2048) 75 us and 81, (512) 43 and 35; 96 (2048) 70 and 80, (1024) 45 and 50, (512) 40
// and 34; 80 (6144) 137 and 149, (4096) 101 and 112 or 114 and 105, (2048) 69 and
// 68; 64 (24576) 357 and 361, (4096) 83 and 78, prompt chunks of 64 (9726) 175 and 185,
// (5119) 146 and 127; between 8192 and 16384 either may win. 256 features have no
// room for them.
// Splits of the token axis: two blocks run at once on a compute unit, one of 256
// features (2048 tokens of 16 heads: 105 us when taken for two, 88 us).
// For few rows, one round of them when there is little else to run, and chunks
// of at most kMaxChunk, which evens out sequences of different lengths (16 of up
// to 4096 tokens and 64 of grouped heads: 65 and 122 us, with 4096 65 and 129, with
// 1024 63 and 131). For many rows, whose queries cost a block about as much as 512
// tokens do, only as many as fill one round (chunks of a quarter of that: 48 heads
// of 4096 tokens 325 us against 261, a step of prompt chunks 240 against 195).
Plan plan(const KvArgs& a, int q_heads) {
  constexpr int64_t kMinChunk = 4 * kGroup, kMaxChunk = 2048;
  const int64_t resident = (a.head_dim <= 128 ? 2 : 1) * 256;
  Plan p;
  p.group = q_heads / a.kv_heads;
  const int64_t rows = (int64_t)a.max_tokens * p.group;
  const auto share = [&](int tile_rows) {   // the tokens that each resident block would take
    p.tile_rows = tile_rows;
    p.tiles = (int)((rows + tile_rows - 1) / tile_rows);
    const int64_t blocks = std::min<int64_t>(most_tiles(a, p) * a.kv_heads, INT32_MAX);
    return (int64_t)a.len_cap * std::max<int64_t>(blocks, 1) / resident;
  };
  const int64_t len = (int64_t)a.len_cap + kGroup;   // a span starts at a whole group
  int64_t chunk;
  p.shared = rows > (a.head_dim <= 128 ? 3 : 2) * kRows;
  p.wide = p.shared && a.head_dim <= 128 && share(128) >= (a.head_dim == 64 ? 8192 : a.head_dim == 80 ? 4096 : 1024);
  if (p.shared)
    chunk = std::min(len, std::max(share(p.wide || a.head_dim == 256 ? 128 : 64), 2 * kMinChunk));
  else
    chunk = std::min(std::max(share(kRows), kMinChunk), kMaxChunk);
  chunk = std::max(chunk, len / kMaxSplits + 1);
  chunk = (chunk + kGroup - 1) / kGroup * kGroup;
  p.chunk = (int)chunk;
  p.splits = (int)((len + chunk - 1) / chunk);
  return p;
}

// The kernel for many rows, kR a wave.
template <int D, int kR>
hipError_t launch_tiles(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t, const Plan& p,
                        hipStream_t s) {
  typedef TileCfg<D, kR> Cfg;
  if (p.tile_rows != Cfg::kBlockRows) return hipErrorInvalidValue;
  // (without cu_tokens every row belongs to a sequence)
  const int64_t jobs = a.num_seqs <= kWave && !a.cu_tokens
                           ? most_tiles(a, p)
                           : first_slot<Cfg::kBlockRows>(a.total_tokens, p.group, a.num_seqs);
  const int64_t blocks = jobs * p.splits * a.kv_heads;
  if (blocks > UINT32_MAX / Cfg::kThreads) return hipErrorInvalidValue;
  if (t.slopes)
    k_kv_attn_tile<D, kR, true><<<(uint32_t)blocks, Cfg::kThreads, 0, s>>>(
        a, r, t, p.group, p.splits, p.chunk);
  else
    k_kv_attn_tile<D, kR, false><<<(uint32_t)blocks, Cfg::kThreads, 0, s>>>(
        a, r, t, p.group, p.splits, p.chunk);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t, hipStream_t s) {
  const Plan p = plan(a, t.q_heads);
  hipError_t e;
  if (p.shared) {
    if constexpr (D <= 128)
      e = p.wide ? launch_tiles<D, 32>(a, r, t, p, s) : launch_tiles<D, 16>(a, r, t, p, s);
    else
      e = launch_tiles<D, 16>(a, r, t, p, s);
  } else {
    const dim3 grid((uint32_t)(p.tiles * a.kv_heads), (uint32_t)a.num_seqs, (uint32_t)p.splits);
    if (t.slopes)
      k_kv_attn_rows<D, true><<<grid, kBlockThreads, 0, s>>>(a, r, t, p.group, p.tiles, p.splits,
                                                             p.chunk);
    else
      k_kv_attn_rows<D, false><<<grid, kBlockThreads, 0, s>>>(a, r, t, p.group, p.tiles, p.splits,
                                                              p.chunk);
    e = hipGetLastError();
  }
  if (e != hipSuccess || p.splits <= 1) return e;
  const int64_t rows = (int64_t)a.total_tokens * t.q_heads;
  if (p.splits <= kFewSplits) {
    constexpr int kBlockRows = kBlockThreads / kWave * (kWave / (D / 4));
    if (rows > (int64_t)INT32_MAX * kBlockRows) return hipErrorInvalidValue;
    k_kv_attn_join_few<D><<<(uint32_t)((rows + kBlockRows - 1) / kBlockRows), kBlockThreads, 0, s>>>(
        t.part, rows, p.splits, t.out);
  } else {
    if (rows > INT32_MAX) return hipErrorInvalidValue;
    k_kv_attn_join<D><<<(uint32_t)rows, kBlockThreads, 0, s>>>(t.part, rows, p.splits, t.out);
  }
  return hipGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(const KvArgs& a, int q_heads) {
  const Plan p = plan(a, q_heads);
  if (p.splits <= 1) return 0;
  return (size_t)a.total_tokens * q_heads * (p.splits * ((int64_t)a.head_dim + 2) + 1) * sizeof(float);
}

hipError_t launch_kv_attention(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t,
                               hipStream_t s) {
  switch (a.head_dim) {
    case 64: return launch_d<64>(a, r, t, s);
    case 80: return launch_d<80>(a, r, t, s);
    case 96: return launch_d<96>(a, r, t, s);
    case 128: return launch_d<128>(a, r, t, s);
    default: return launch_d<256>(a, r, t, s);
  }
}

}  // namespace i8mm
