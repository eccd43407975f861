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
// the cache and sum the product exactly. An fp16 MFMA would have half the rate
// and need the codes converted; 15 bits are finer than the fp16 the query came
// in for all but the smallest features of a row.
//
// Softmax in base 2 with the running maximum m of each row. The value absmax
// is folded into the weight: P = 2^(S - m + log2 r), r = absmax / ref, for one
// ref a wave; O is then in units of ref / 127 and the row sum takes P / r.
// P <= 2^kLazy is rounded to fp16 (2^-11 relative; below 2^-14 of the row's
// maximum, 2^-25 absolute); all sums are fp32.

#include <algorithm>

#include "kv_common.h"

namespace i8mm {

namespace {

constexpr int kGroup = 64;          // tokens of a step: four blocks
constexpr int kRows = 16;           // rows of a tile
constexpr float kLazy = 8.f;        // a row is rescaled when its maximum grew by more
constexpr float kMinRatio = 0x1p-40f;   // weights of such values vanish in fp16 anyway

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

__device__ __forceinline__ float max_over_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
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

// The row's query as the B operand: lane (row, g) holds features 64 c + 16 g ..
// + 15 of it, zero past D. Returns a / 16256.
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* row, int pos, bool live,
                                            const RotaryArgs& rot, int g, v4i32* hi, v4i32* lo) {
  constexpr int kC = (D + 63) / 64;
  float x[kC][16];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e0 = 64 * c + 16 * g;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[c][e] = 0.f;
    if (live && e0 < D) {
      load8_rotated(row, e0, pos, rot, x[c]);
      load8_rotated(row, e0 + 8, pos, rot, x[c] + 8);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t m = __builtin_bit_cast(uint32_t, x[c][e]) & 0x7fffffffu;
      top = top > m ? top : m;
    }
  }
  uint32_t o = (uint32_t)__shfl_xor((int)top, 16, kWave);
  top = top > o ? top : o;
  o = (uint32_t)__shfl_xor((int)top, 32, kWave);
  top = top > o ? top : o;
  if (top <= 0x08000000u) top = 0;   // 2^-111: 16256 / a stays finite
  const float a = __builtin_bit_cast(float, top);
  const float s = top ? 16256.0f / a : 0.f;
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t ph = 0, pl = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = (int)rintf(x[c][4 * w + i] * s);
        const int h = (q + 64) >> 7;
        ph |= ((uint32_t)h & 0xffu) << (8 * i);
        pl |= ((uint32_t)(q - (h << 7)) & 0xffu) << (8 * i);
      }
      hi[c][w] = (int)ph;
      lo[c][w] = (int)pl;
    }
  return a / 16256.0f;
}

// A wave's blocks: lane 4 i + j holds block j of its i-th group.
struct BlockList {
  int lin;            // -1 where there is no block to read
  float ks;           // key absmax / 127
  float log_r, inv_r; // of the value absmax over the wave's ref
};

// ---- Codes through LDS. A group is staged as its four blocks, each as it lies
// in the cache, kPitch apart: 64 bytes more than a block, so that the four
// blocks a key operand touches lie in different banks. Staging is LDS-DMA, 1 KB
// an instruction, with no registers in between; the waits count its
// instructions, so each stage issues the same number of them.
typedef __attribute__((address_space(3))) void* lds_ptr_t;

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
__device__ __forceinline__ void read_keys(const int8_t* st, int n, int g,
                                          v4i32 (&k)[(D + 63) / 64][4]) {
  const int8_t* p = st + (n >> 2) * Stage<D>::kPitch + (n & 3) * 16;
#pragma unroll
  for (int c = 0; c < (D + 63) / 64; ++c) {
    const int8_t* pc = p + min(4 * c + g, D / 16 - 1) * kTile;
#pragma unroll
    for (int q = 0; q < 4; ++q) k[c][q] = *reinterpret_cast<const v4i32*>(pc + q * 64);
  }
}
// Its values: feature 16 d + n, the 16 tokens of block g.
template <int D>
__device__ __forceinline__ v4i32 read_values(const int8_t* st, int n, int g, int d) {
  return *reinterpret_cast<const v4i32*>(st + g * Stage<D>::kPitch + d * kTile + n * 16);
}

// One column tile's scores of a group, S^T = K Q^T as integers: element e of a
// lane is (e >> 2, e & 3) of s.
template <int D>
__device__ __forceinline__ void scores(const v4i32 (&k)[(D + 63) / 64][4], const v4i32* qh,
                                       const v4i32* ql, v4i32 (&s)[4]) {
  constexpr int kC = (D + 63) / 64;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    s[q] = v4i32{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < kC; ++c)
      s[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[c][q], qh[c], s[q],
                                                   0, 0, 0);
    s[q] = s[q] << 7;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      s[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[c][q], ql[c], s[q],
                                                   0, 0, 0);
  }
}

// A lane's row: its position, visible tokens and factors.
struct Row {
  int pos, lo, hi;
  float qf;      // query absmax / 16256 * scale * log2(e)
  float slope;   // * log2(e)
};

// Logits of a group in base 2, hidden ones -infinity.
template <bool kAlibi>
__device__ __forceinline__ void logits(const v4i32 (&s)[4], const Row& row, float ks, int t0, int g,
                                       bool masked, bool here, float (&z)[16]) {
  const float f = ks * row.qf;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    z[e] = (float)s[e >> 2][e & 3] * f;
    if (kAlibi) z[e] += row.slope * (float)(t0 + 16 * g + e - row.pos);
  }
  if (masked) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int tok = t0 + 16 * g + e;
      if (!here || tok < row.lo || tok >= row.hi) z[e] = -INFINITY;
    }
  }
}

// The running maximum over a group's logits: true (the whole wave) when rows
// are to be rescaled, each by its alpha.
__device__ __forceinline__ bool new_maximum(const float (&z)[16], float* m, float* alpha) {
  float top = z[0];
#pragma unroll
  for (int e = 1; e < 16; ++e) top = fmaxf(top, z[e]);
  top = max_over_groups(top);
  if (!__any(top > *m + kLazy)) return false;
  const float next = fmaxf(*m, top);
  *alpha = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(*m - next);
  *m = next;
  return true;
}

// ---- Few rows: each wave streams its own groups through its own part of
// LDS, keys and values apart: a buffer is refilled as soon as it has been read,
// so something is always in flight. The four waves of a block join through LDS,
// the blocks of a row tile through the workspace and k_kv_attn_join.
template <int D, bool kAlibi>
__global__ __launch_bounds__(kBlockThreads) void k_kv_attn_rows(KvArgs a, RotaryArgs rot,
                                                                AttnArgs t, int group, int tiles,
                                                                int splits, int chunk) {
  constexpr int kC = (D + 63) / 64, kT = D / 16, kLd = D + 4;
  typedef Stage<D> S;
  constexpr int kSlots = D <= 64 ? 2 : 1;
  constexpr int kAhead = (2 * kSlots - 1) * 4 * S::kLoads;   // loads younger than the awaited
  constexpr int kJoinBytes = (4 * kRows * kLd + 8 * kRows) * 4;
  constexpr int kStageBytes = 4 * 2 * kSlots * S::kGroupBytes;
  __shared__ __attribute__((aligned(1024)))
  int8_t lds[kStageBytes > kJoinBytes ? kStageBytes : kJoinBytes];
  float(*s_o)[kRows][kLd] = reinterpret_cast<float(*)[kRows][kLd]>(lds);
  float(*s_m)[kRows] = reinterpret_cast<float(*)[kRows]>(lds + 4 * kRows * kLd * 4);
  float(*s_l)[kRows] = s_m + 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, h = blockIdx.y / tiles, b = blockIdx.z;
  const int r_first = (blockIdx.y % tiles) * kRows;
  const KvSeq sq = kv_seq(a, b);
  const int rows = sq.n * group;
  if (r_first >= rows) return;
  const int r_last = min(r_first + kRows, rows) - 1;
  const Span span = row_span(t, sq, r_first / group, r_last / group);
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
  v4i32 qh[kC], ql[kC];
  const uint16_t* q_row = t.q + (int64_t)(sq.row0 + i_row) * t.q_ts + (int64_t)head * t.q_hs;
  row.qf = load_query<D>(q_row, max(row.pos, 0), live && row.pos >= 0, rot, g, qh, ql) * t.scale_log2;
  row.lo = visible_lo(t, row.pos);
  row.hi = live ? visible_hi(t, sq, row.pos) : 0;
  row.slope = kAlibi ? t.slopes[head] * 1.44269504088896340736f : 0.f;
  // groups inside [all_lo, all_hi) are visible to every row
  const int all_lo = visible_lo(t, sq.first + r_last / group);
  const int all_hi = visible_hi(t, sq, sq.first + r_first / group);

  v4f32 o[kT];
#pragma unroll
  for (int d = 0; d < kT; ++d) o[d] = v4f32{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f, ref = 0.f;

  const int gi_end = (end + kGroup - 1) / kGroup;
  for (int gi0 = begin / kGroup + wave; gi0 < gi_end; gi0 += 64) {
    BlockList bl;
    bl.lin = -1;
    bl.ks = 0.f;
    float v_absmax = 0.f;
    {
      const int gi = gi0 + 4 * (lane >> 2), blk = 4 * gi + (lane & 3);
      if (gi < gi_end && blk * kKvBlock < end) bl.lin = kv_block(a, b, h, blk);
      if (bl.lin >= 0) {
        bl.ks = a.k_absmax[bl.lin] / 127.0f;
        v_absmax = a.v_absmax[bl.lin];
      }
    }
    const uint64_t present = __ballot(bl.lin >= 0);
    const int count = min(16, (gi_end - gi0 + 3) / 4);
    // absent blocks are masked; block 0 is read in their place
    auto load = [&](int i, const int8_t* codes, int8_t* dst) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        stage_block<D>(codes, max(__builtin_amdgcn_readlane(bl.lin, 4 * i + j), 0),
                       dst + j * S::kPitch, lane);
    };
    auto step = [&](int i, int8_t* ks, int8_t* vs) __attribute__((always_inline)) {
      const uint32_t have = (uint32_t)(present >> (4 * i)) & 15u;
      const int t0 = (gi0 + 4 * i) * kGroup;
      v4i32 s[4];
      float z[16], alpha;
      if (i + kSlots < count) wait_loads<kAhead>(); else wait_loads<0>();
      {
        v4i32 kf[kC][4];
        read_keys<D>(ks, n, g, kf);
        scores<D>(kf, qh, ql, s);
      }
      if (i + kSlots < count) {
        wait_lds_reads();
        load(i + kSlots, a.k_codes, ks);
      }
      logits<kAlibi>(s, row, __shfl(bl.ks, 4 * i + g, kWave), t0, g,
                     t0 < all_lo || t0 + kGroup > all_hi || have != 15u, (have >> g) & 1u, z);
      if (new_maximum(z, &m, &alpha)) {
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kT; ++d) o[d] *= alpha;
      }
      const float off = (m == -INFINITY ? 0.f : m) - __shfl(bl.log_r, 4 * i + g, kWave);
      float sum = 0.f;
      uint32_t ph[8], pl[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p0 = __builtin_amdgcn_exp2f(z[2 * e] - off);
        const float p1 = __builtin_amdgcn_exp2f(z[2 * e + 1] - off);
        sum += p0 + p1;
        ph[e] = f2h2(p0, p1);
        pl[e] = f2h2(p0 - h2f(ph[e] & 0xffffu), p1 - h2f(ph[e] >> 16));
      }
      l += sum * __shfl(bl.inv_r, 4 * i + g, kWave);
      const v8f16 p0h = __builtin_bit_cast(v8f16, make_uint4(ph[0], ph[1], ph[2], ph[3]));
      const v8f16 p1h = __builtin_bit_cast(v8f16, make_uint4(ph[4], ph[5], ph[6], ph[7]));
      const v8f16 p0l = __builtin_bit_cast(v8f16, make_uint4(pl[0], pl[1], pl[2], pl[3]));
      const v8f16 p1l = __builtin_bit_cast(v8f16, make_uint4(pl[4], pl[5], pl[6], pl[7]));
      if (i + kSlots < count) wait_loads<kAhead>(); else wait_loads<0>();
#pragma unroll
      for (int d = 0; d < kT; ++d) {
        v8f16 v0, v1;
        codes_to_f16(read_values<D>(vs, n, g, d), &v0, &v1);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0l, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1l, o[d], 0, 0, 0);
      }
      if (i + kSlots < count) {
        wait_lds_reads();
        load(i + kSlots, a.v_codes, vs);
      }
    };
    int8_t* const st_k = lds + wave * (2 * kSlots * S::kGroupBytes);
    int8_t* const st_v = st_k + kSlots * S::kGroupBytes;
    wait_lds_reads();   // of an earlier list's last groups
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (i < count) {
        load(i, a.k_codes, st_k + i * S::kGroupBytes);
        load(i, a.v_codes, st_v + i * S::kGroupBytes);
      }
    {
      float top = v_absmax;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
      if (top > ref) {
        const float f = ref / top;
#pragma unroll
        for (int d = 0; d < kT; ++d) o[d] *= f;
        ref = top;
      }
      float ratio = v_absmax / (ref > 0.f ? ref : 1.f);
      ratio = ratio < kMinRatio ? kMinRatio : ratio;   // (keeps a NaN)
      bl.log_r = __builtin_amdgcn_logf(ratio);
      bl.inv_r = 1.0f / ratio;
    }
    for (int i = 0; i < count; ++i) {
      const int slot = kSlots == 1 ? 0 : i % kSlots;
      step(i, st_k + slot * S::kGroupBytes, st_v + slot * S::kGroupBytes);
    }
  }

  // join the four waves
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  __syncthreads();   // every wave is done with the staged groups
  const float unit = ref / 127.0f;
#pragma unroll
  for (int d = 0; d < kT; ++d) *reinterpret_cast<v4f32*>(&s_o[wave][n][16 * d + 4 * g]) = o[d] * unit;
  if (g == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
  }
  __syncthreads();
  const int64_t part_rows = (int64_t)a.total_tokens * t.q_heads;
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
      const float inv = total == 0.f ? 0.f : 1.0f / total;
      *reinterpret_cast<uint2*>(t.out + out_row * D + d4) =
          make_uint2(f2h2(acc[0] * inv, acc[1] * inv), f2h2(acc[2] * inv, acc[3] * inv));
    } else {
      const int64_t part = split * part_rows + out_row;
      *reinterpret_cast<v4f32*>(t.part + part * D + d4) = acc;
      if (d4 == 0) {
        float* ml = t.part + (int64_t)splits * part_rows * D + part * 2;
        ml[0] = top;
        ml[1] = total;
      }
    }
  }
}

// One wave a row: the splits' sums, weighed by their maxima.
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_attn_join(KvArgs a, AttnArgs t, int group,
                                                                int splits, int chunk) {
  constexpr int kE = (D + 63) / 64;
  const int lane = threadIdx.x & 63;
  const int r = blockIdx.x * (kBlockThreads / kWave) + (threadIdx.x >> 6);
  const int h = blockIdx.y, b = blockIdx.z;
  const KvSeq sq = kv_seq(a, b);
  const int rows = sq.n * group;
  if (r >= rows) return;
  const int tile = r / kRows * kRows;
  const Span span = row_span(t, sq, tile / group, (min(tile + kRows, rows) - 1) / group);
  if (span.end - span.begin <= chunk) return;   // written by its only split
  const int parts = (span.end - span.begin + chunk - 1) / chunk;
  const int64_t part_rows = (int64_t)a.total_tokens * t.q_heads;
  const int64_t row = (int64_t)(sq.row0 + r / group) * t.q_heads + h * group + r % group;
  const float* ml = t.part + (int64_t)splits * part_rows * D;
  float top = -INFINITY;
  for (int p = lane; p < parts; p += kWave) top = fmaxf(top, ml[(p * part_rows + row) * 2]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[kE], total = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
  for (int p = 0; p < parts; ++p) {
    const int64_t part = p * part_rows + row;
    const float w = __builtin_amdgcn_exp2f(ml[part * 2] - base);
    total += ml[part * 2 + 1] * w;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int d = e * kWave + lane;
      if (d < D) acc[e] += t.part[part * D + d] * w;
    }
  }
  const float inv = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int d = e * kWave + lane;
    if (d < D) t.out[row * D + d] = f2h(acc[e] * inv);
  }
}

struct Plan {
  int group, tiles, splits, chunk;
};

// Splits of the token axis so that about four blocks a compute unit run, none
// shorter than a group for each wave.
Plan plan(const KvArgs& a, int q_heads) {
  constexpr int64_t kBlocks = 4 * 256, kMinChunk = 4 * kGroup;
  Plan p;
  p.group = q_heads / a.kv_heads;
  p.tiles = (int)(((int64_t)a.max_tokens * p.group + kRows - 1) / kRows);
  const int64_t items = std::max<int64_t>((int64_t)p.tiles * a.kv_heads * a.num_seqs, 1);
  const int64_t want = std::max<int64_t>((kBlocks + items - 1) / items, 1);
  const int64_t len = std::max<int64_t>(a.len_cap, 1) + kGroup;   // a span starts at a whole group
  int64_t chunk = (len + want - 1) / want;
  chunk = (std::max(chunk, kMinChunk) + kGroup - 1) / kGroup * kGroup;
  p.chunk = (int)chunk;
  p.splits = (int)((len + chunk - 1) / chunk);
  return p;
}

}  // namespace

size_t attn_workspace_bytes(const KvArgs& a, int q_heads) {
  const Plan p = plan(a, q_heads);
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * a.total_tokens * q_heads * (a.head_dim + 2) * sizeof(float);
}

template <int D>
hipError_t launch_d(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t, hipStream_t s) {
  const Plan p = plan(a, t.q_heads);
  const int64_t y = (int64_t)p.tiles * a.kv_heads;
  if (y > 65535) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)p.splits, (uint32_t)y, (uint32_t)a.num_seqs);
  if (t.slopes)
    k_kv_attn_rows<D, true><<<grid, kBlockThreads, 0, s>>>(a, r, t, p.group, p.tiles, p.splits, p.chunk);
  else
    k_kv_attn_rows<D, false><<<grid, kBlockThreads, 0, s>>>(a, r, t, p.group, p.tiles, p.splits, p.chunk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits <= 1) return e;
  const dim3 join((uint32_t)(((int64_t)a.max_tokens * p.group + 3) / 4), (uint32_t)a.kv_heads,
                  (uint32_t)a.num_seqs);
  k_kv_attn_join<D><<<join, kBlockThreads, 0, s>>>(a, t, p.group, p.splits, p.chunk);
  return hipGetLastError();
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
