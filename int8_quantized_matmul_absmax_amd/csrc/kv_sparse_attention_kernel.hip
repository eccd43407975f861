// Attention over chosen pages of the paged 8-bit key/value cache.
//
// Each token and key/value head has its own list of pages, so its rows are only the
// query heads that share the head. The arithmetic is the dense kernels', the weights
// in two parts of fp16 as for few rows. A list's tokens are counted on from page to
// page: groups of 64 of them may begin inside one page and end in another.

#include "kv_attention_common.h"

namespace i8mm {

namespace {

// Entries of a list up to the last page that may be visible.
__device__ __forceinline__ int entries_of(const int32_t* list, int count, int seen_pages, int lane) {
  int entries = 0;
  for (int e0 = 0; e0 < count; e0 += kWave) {
    const int e = e0 + lane;
    const uint64_t there = __ballot(e < count && (uint32_t)list[min(e, count - 1)] < (uint32_t)seen_pages);
    if (there) entries = e0 + 64 - __builtin_clzll(there);
  }
  return entries;
}

// ---- Few tokens: a block takes up to 16 rows, its four waves share a list, and a list
// may be split. 64 tokens with lists of 64 pages of 16 tokens, 64 heads on 8 of 128
// features (131 MB): 25.8 us, 5.1 TB/s; one token, 16 pages of 128 tokens, 32 heads on
// 8: 7.8 us and 3.6 to join.
template <int D>
__global__ __launch_bounds__(kBlockThreads, D <= 128 ? 2 : 1) void k_kv_attn_pages(
    KvArgs a, RotaryArgs rot, AttnArgs t, const int32_t* chosen, int count, int group, int tiles,
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
  // heads first: blocks go to the 8 XCDs in turn, and a head's share an L2
  const int per_token = a.kv_heads * tiles * splits;
  const int token = blockIdx.x / per_token, job = blockIdx.x % per_token;
  const int h = job % a.kv_heads, tile = job / a.kv_heads % tiles, split = job / a.kv_heads / tiles;
  const int r_first = tile * kRows, r_last = min(r_first + kRows, group) - 1;
  const int b = sequence_of(a, token, lane);
  const KvSeq sq = kv_seq(a, b);
  const int i = token - sq.row0;
  // (a token of no sequence, or before one, sees nothing)
  const bool belongs = i >= 0 && i < sq.n && sq.first + i >= 0;
  const int pos = belongs ? sq.first + i : 0;
  const int64_t out_row0 = (int64_t)token * t.q_heads + h * group;
  const Parts parts = parts_of(t.part, (int64_t)a.total_tokens * t.q_heads, splits, D);

  const int32_t* const list = chosen + ((int64_t)token * a.kv_heads + h) * count;
  const int page_tokens = a.slots * kKvBlock;
  const int seen_pages = belongs ? pos / page_tokens + 1 : 0;
  const int entries = entries_of(list, count, seen_pages, lane);
  const int all = entries * page_tokens;
  // (the last takes what is left: of a list longer than its sequence, then)
  const int begin = split * chunk, end = split == splits - 1 ? all : min(begin + chunk, all);
  const bool only = splits == 1 || all <= chunk;
  if (split > 0 && begin >= all) return;

  const bool live = r_first + n <= r_last;
  constexpr int kPasses = (kRows + 4 * Q::kPassRows - 1) / (4 * Q::kPassRows);
  QueryLoads q_in[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = min(r_first + (4 * p + wave) * Q::kPassRows + lane / Q::kLanes, r_last);
    load_query<D>(t.q + (int64_t)token * t.q_ts + (int64_t)(h * group + rr) * t.q_hs, pos, rot, t.q,
                  lane, q_in[p]);
  }
  v4i32 qh[kC], ql[kC];
  Row row;
  row.pos = pos;
  row.lo = 0;
  row.slope = 0.f;
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
  int room;   // tokens of a list's block that are visible
  auto load = [&](int i, const int8_t* codes, int8_t* dst) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      stage_block<D>(codes, max(__builtin_amdgcn_readlane(bl.lin, 4 * i + j), 0),
                     dst + j * S::kPitch, lane);
  };
  // the list of 16 groups from gi0 on, and the first group's copies
  auto start = [&](int gi0) __attribute__((always_inline)) {
    bl.lin = -1;
    k_absmax = v_absmax = 0.f;
    room = 0;
    const int c = 4 * (gi0 + 4 * (lane >> 2)) + (lane & 3);
    if (c * kKvBlock < end) {
      const int e = c / a.slots, page = list[e];
      if ((uint32_t)page < (uint32_t)seen_pages) {
        const int blk = page * a.slots + (c - e * a.slots);
        room = min(pos + 1 - blk * kKvBlock, kKvBlock);
        if (room > 0) bl.lin = kv_block(a, b, h, blk);
      }
    }
    if (bl.lin >= 0) {
      k_absmax = a.k_absmax[bl.lin];
      v_absmax = a.v_absmax[bl.lin];
    } else {
      room = 0;
    }
    load(0, a.k_codes, st_k);
    load(0, a.v_codes, st_v);
  };
  if (gi_first < gi_end) start(gi_first);
  float x_in[kPasses][16];
  uint32_t x_top[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = r_first + (4 * p + wave) * Q::kPassRows + lane / Q::kLanes;
    x_top[p] = rotate_query<D>(q_in[p], r <= r_last && belongs, rot, lane, x_in[p]);
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
    const uint64_t whole = __ballot(room == kKvBlock);
    const int groups = min(16, (gi_end - gi0 + 3) / 4);
    list_factors(k_absmax, v_absmax, &bl);
    for (int i = 0; i < groups; ++i) {
      v4i32 s[4];
      float x[16], p[16];
      if (i + 1 < groups) wait_loads<kAhead>(); else wait_loads<0>();
      scores<D>(st_k, n, g, qh, ql, s);
      if (i + 1 < groups) {
        wait_lds_reads();
        load(i + 1, a.k_codes, st_k);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = (float)s[e >> 2][e & 3];
      Scale sc = {__shfl(bl.ks, 4 * i + g, kWave), __shfl(bl.log_a, 4 * i + g, kWave),
                  __shfl(bl.inv_a, 4 * i + g, kWave)};
      // (a lane's block begins at its own token 0)
      const int here = __shfl(room, 4 * i + g, kWave);
      row.hi = live ? here : 0;
      const float top = max_over_groups<4>(logits<false>(
          x, &sc, row, -16 * g, g, ((uint32_t)(whole >> (4 * i)) & 15u) != 15u, true));
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
      if (i + 1 < groups) wait_loads<kAhead>(); else wait_loads<0>();
#pragma unroll
      for (int d = 0; d < kT; ++d) {
        v8f16 v0, v1;
        codes_to_f16(read_values<D>(st_v, n, g, d), &v0, &v1);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1h, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0l, o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1l, o[d], 0, 0, 0);
      }
      if (i + 1 < groups) {
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
    const int64_t out_row = out_row0 + r_first + row;
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
    if (splits > 1 && split == 0 && d4 == 0) parts.count[out_row] = min((all + chunk - 1) / chunk, splits);
  }
}

// ---- Many tokens: a wave takes a token and head by itself, and nothing is joined.
// Bound by the vector pipe (exponentials, conversions), of whose lanes a group of four
// query heads would use a quarter: so kCls groups of 64 tokens are done at once, each
// with 16 / kCls of the MFMA's columns. A group's products take queries and weights
// that are zero outside its own columns, so scores of all of them add up in one set of
// registers, and a column's sums are those of every kCls-th group, with a maximum and a
// row sum of its own. The columns of a row are joined at the end.
//
// A wave's stages, keys of kCls groups and then their values, go through two buffers
// of its part of LDS, each refilled as soon as it has been read (with 64 features
// three and four take the room of a third block a compute unit: 176 and 179 us, so 154).
//
// 1367 tokens with lists of 32 pages of 48 tokens, 32 heads on 8 of 64 features (what
// the lists name, 3.2 GB, comes from the L2s): traced 154 us (a pass among others 135, 24
// TB/s), against 216 by the kernel above; of 128 features 284 us, 23 TB/s, against 387:
// what the L2s give.
template <int D, int kCls>
struct WaveCfg {
  typedef Stage<D> S;
  static constexpr int kCols = kRows / kCls;
  static constexpr int kWaves = 4;
  static constexpr int kStageLoads = 4 * S::kLoads;
  static constexpr int kQueryBytes = kCols * (QueryCfg<D>::kRowBytes + 16);
  static constexpr int kBuffers = 2;
  static constexpr int kWaveBytes = (kBuffers * S::kGroupBytes + kQueryBytes + 15) / 16 * 16;
};

template <int D, int kCls>
__global__ __launch_bounds__(kBlockThreads, D == 64 ? 3 : D <= 128 ? 2 : 1) void k_kv_attn_pages_wave(
    KvArgs a, RotaryArgs rot, AttnArgs t, const int32_t* chosen, int count, int group) {
  typedef WaveCfg<D, kCls> Cfg;
  typedef Stage<D> S;
  typedef QueryCfg<D> Q;
  constexpr int kC = (D + 63) / 64, kT = D / 16, kCols = Cfg::kCols, kBuffers = Cfg::kBuffers;
  constexpr int kAhead = (kBuffers - 1) * Cfg::kStageLoads;
  constexpr int kListGroups = 16;
  __shared__ __attribute__((aligned(1024))) int8_t lds[Cfg::kWaves * Cfg::kWaveBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4, cls = n / kCols, r = n % kCols;
  // heads first: blocks go to the 8 XCDs in turn, and a head's share an L2
  const int h = blockIdx.x % a.kv_heads, token = blockIdx.x / a.kv_heads * Cfg::kWaves + wave;
  if (token >= a.total_tokens) return;
  int8_t* const ring = lds + wave * Cfg::kWaveBytes;
  int8_t* const lds_q = ring + kBuffers * S::kGroupBytes;
  float* const s_qf = reinterpret_cast<float*>(lds_q + kCols * Q::kRowBytes);
  const int b = sequence_of(a, token, lane);
  const KvSeq sq = kv_seq(a, b);
  const int i_token = token - sq.row0;
  // (a token of no sequence, or before one, sees nothing)
  const bool belongs = i_token >= 0 && i_token < sq.n && sq.first + i_token >= 0;
  const int pos = belongs ? sq.first + i_token : 0;
  const int32_t* const list = chosen + ((int64_t)token * a.kv_heads + h) * count;
  const int seen_pages = belongs ? pos / (a.slots * kKvBlock) + 1 : 0;
  const int entries = entries_of(list, count, seen_pages, lane);
  const int blocks = entries * a.slots, groups = (blocks + 3) / 4;

  // the queries: columns past the group's rows repeat the last
  constexpr int kPasses = (kCols + Q::kPassRows - 1) / Q::kPassRows;
  QueryLoads q_in[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = min(p * Q::kPassRows + lane / Q::kLanes, group - 1);
    load_query<D>(t.q + (int64_t)token * t.q_ts + (int64_t)(h * group + rr) * t.q_hs, pos, rot, t.q,
                  lane, q_in[p]);
  }
  float x_in[kPasses][16];
  uint32_t x_top[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) x_top[p] = rotate_query<D>(q_in[p], belongs, rot, lane, x_in[p]);
  row_absmax<D>(x_top);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int rr = p * Q::kPassRows + lane / Q::kLanes;
    if (rr < kCols) store_query<D>(x_in[p], x_top[p], rot, lane, lds_q + rr * Q::kRowBytes, s_qf + rr);
  }
  wait_lds_reads();   // (the wave's own stores)
  v4i32 qh[kC], ql[kC];
  read_query<D>(lds_q + r * Q::kRowBytes, g, qh, ql);
  Row row;
  row.pos = pos;
  row.lo = 0;
  row.slope = 0.f;
  row.qf = s_qf[r] * t.scale_log2;

  v4f32 o[kT];
#pragma unroll
  for (int d = 0; d < kT; ++d) o[d] = v4f32{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  for (int gi0 = 0; gi0 < groups; gi0 += kListGroups) {
    // lane 4 i + j: block j of group gi0 + i
    BlockList bl;
    float k_absmax = 0.f, v_absmax = 0.f;
    int room = 0;   // tokens of the block that are visible
    bl.lin = -1;
    const int c = 4 * gi0 + lane;
    if (c < blocks) {
      const int e = c / a.slots, page = list[e];
      if ((uint32_t)page < (uint32_t)seen_pages) {
        const int blk = page * a.slots + (c - e * a.slots);
        room = max(min(pos + 1 - blk * kKvBlock, kKvBlock), 0);
        if (room > 0) bl.lin = kv_block(a, b, h, blk);
      }
    }
    if (bl.lin >= 0) {
      k_absmax = a.k_absmax[bl.lin];
      v_absmax = a.v_absmax[bl.lin];
    } else {
      room = 0;
    }
    const uint64_t whole = __ballot(room == kKvBlock);
    const int sets = (min(kListGroups, groups - gi0) + kCls - 1) / kCls;
    const int stages = sets * 2 * kCls;
    // stage s: of set s / (2 kCls), keys of its kCls groups, then their values; past the
    // last, block 0 again, so that the waits can count
    auto load = [&](int s, int buffer) __attribute__((always_inline)) {
      const int in_set = s % (2 * kCls);
      const int i = s < stages ? s / (2 * kCls) * kCls + in_set % kCls : 0;
      const int8_t* const codes = in_set < kCls ? a.k_codes : a.v_codes;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        stage_block<D>(codes, max(__builtin_amdgcn_readlane(bl.lin, 4 * i + j), 0),
                       ring + buffer * S::kGroupBytes + j * S::kPitch, lane);
    };
    int s = 0, buffer = 0;
#pragma unroll
    for (int u = 0; u < kBuffers; ++u) load(u, u);
    list_factors(k_absmax, v_absmax, &bl);
    auto next = [&]() __attribute__((always_inline)) {
      wait_lds_reads();
      load(s + kBuffers, buffer);
      ++s;
      buffer = buffer + 1 == kBuffers ? 0 : buffer + 1;
    };
    for (int set = 0; set < sets; ++set) {
      v4i32 hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) hi[q] = lo[q] = v4i32{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kCls; ++k) {
        const int mine = cls == k ? -1 : 0;
        const int8_t* const st = ring + buffer * S::kGroupBytes;
        wait_loads<kAhead>();
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v4i32 keys = read_keys<D>(st, n, g, c, q);
            hi[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(keys, qh[c] & mine, hi[q], 0, 0, 0);
            lo[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(keys, ql[c] & mine, lo[q], 0, 0, 0);
          }
        next();
      }
      float x[16], p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = (float)((hi[e >> 2][e & 3] << 7) + lo[e >> 2][e & 3]);
      const int at = 4 * (set * kCls + cls) + g;
      Scale sc = {__shfl(bl.ks, at, kWave), __shfl(bl.log_a, at, kWave), __shfl(bl.inv_a, at, kWave)};
      row.hi = __shfl(room, at, kWave);
      constexpr uint64_t kAll = (1ull << (4 * kCls)) - 1;
      const bool masked = ((whole >> (4 * kCls * set)) & kAll) != kAll;
      const float top = max_over_groups<4>(logits<false>(x, &sc, row, -16 * g, g, masked, true));
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
      v4i32 ph[2], pl[2];   // the weights in two parts of 11 bits
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = f2h2(p[2 * e], p[2 * e + 1]);
        ph[e >> 2][e & 3] = (int)w;
        pl[e >> 2][e & 3] = (int)f2h2(p[2 * e] - h2f(w & 0xffffu), p[2 * e + 1] - h2f(w >> 16));
      }
#pragma unroll
      for (int k = 0; k < kCls; ++k) {
        const int mine = cls == k ? -1 : 0;
        const int8_t* const st = ring + buffer * S::kGroupBytes;
        const v8f16 p0h = __builtin_bit_cast(v8f16, ph[0] & mine), p1h = __builtin_bit_cast(v8f16, ph[1] & mine);
        const v8f16 p0l = __builtin_bit_cast(v8f16, pl[0] & mine), p1l = __builtin_bit_cast(v8f16, pl[1] & mine);
        wait_loads<kAhead>();
#pragma unroll
        for (int d = 0; d < kT; ++d) {
          v8f16 v0, v1;
          codes_to_f16(read_values<D>(st, n, g, d), &v0, &v1);
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0h, o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1h, o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p0l, o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p1l, o[d], 0, 0, 0);
        }
        next();
      }
    }
    wait_loads<0>();   // (of the next list, or the end: nothing may land in LDS after it)
  }

  // join the row's columns
  float top = m;
#pragma unroll
  for (int d = kCols; d < kRows; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  const float w = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
  l *= w;
#pragma unroll
  for (int d = kCols; d < kWave; d <<= 1) l += __shfl_xor(l, d, kWave);
  const float inv = inverse(l);
  uint16_t* const out = t.out + ((int64_t)token * t.q_heads + h * group + r) * D;
#pragma unroll
  for (int d = 0; d < kT; ++d) {
    v4f32 y = o[d] * w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int x = kCols; x < kRows; x <<= 1) y[e] += __shfl_xor(y[e], x, kWave);
    }
    if (cls == 0 && r < group)
      *reinterpret_cast<uint2*>(out + 16 * d + 4 * g) =
          make_uint2(f2h2(y[0] * inv, y[1] * inv), f2h2(y[2] * inv, y[3] * inv));
  }
}

// The kernel for many tokens from kManyWaves of its waves on, where up to eight query
// heads share a key/value head (lists as above, this one and the one for few): 2048
// waves of 128 features 161 us and 147, 2216 of 64 47 and 50, of 128 96 and 93, 3768
// 83 and 84, 157 and 170, of 256 335 and 382, 5088 of 64, 80 and 128 104 and 115, 152
// and 153, 200 and 220.
constexpr int kManyWaves = 2560;
// Splits of a list's tokens, as for few rows of the dense attention.
struct Plan {
  int group, tiles, splits, chunk;
  bool wave;   // the kernel for many tokens
};
Plan plan(const KvArgs& a, int q_heads, int count) {
  constexpr int64_t kMinChunk = 4 * kGroup, kMaxSplits = 1024;
  const int64_t resident = (a.head_dim <= 128 ? 2 : 1) * 256;
  // Up to two chunks are not worth a join of up to 128 features: 32 rows of 512 tokens of
  // 128 features 8.8 us and 9.6 in two splits, 768 tokens 10.3 and 9.9 in three; of 256
  // features 512 tokens 12.2 and 11.7.
  const int64_t kWhole = a.head_dim <= 128 ? 2 * kMinChunk : kMinChunk;
  Plan p;
  p.group = q_heads / a.kv_heads;
  p.tiles = (p.group + kRows - 1) / kRows;
  p.wave = p.group <= 8 && (int64_t)a.total_tokens * a.kv_heads >= kManyWaves;
  if (p.wave) {
    p.splits = 1;
    p.chunk = 0;
    return p;
  }
  // Tokens of a list: of one that names pages once, no more than its sequence has. (992
  // lists of 129 pages of 48 tokens, of sequences of 92, took 36 us with
  // four splits each; so 16.8.)
  const int64_t tokens = std::min<int64_t>((int64_t)count * a.slots * kKvBlock,
                                           ((int64_t)a.len_cap + kGroup - 1) / kGroup * kGroup);
  const int64_t blocks = (int64_t)a.total_tokens * a.kv_heads * p.tiles;
  // (with blocks for two rounds there is nothing to fill, and sums to join would take
  // room for every one of their rows)
  int64_t chunk = tokens;
  if (blocks < 2 * resident && tokens > kWhole) {
    // (no more splits than are resident at once: 96 blocks of 4096 tokens in six splits
    // 29.5 us, in five 25.6; of 256 features 40 of 4096 in seven 32.0, in six 25.0. Nor for
    // long chunks, however long: cut to 2048 tokens 512 blocks of 8192 take 195 us and
    // whole 185, 1016 377 and 360, of 256 features 160 138 and 121; 320 blocks 125 and 138,
    // which fill the card less well whole)
    const int64_t splits = std::max<int64_t>(resident / std::max<int64_t>(blocks, 1), 1);
    chunk = std::max((tokens + splits - 1) / splits, kMinChunk);
  }
  chunk = std::max(chunk, tokens / kMaxSplits + 1);
  chunk = (chunk + kGroup - 1) / kGroup * kGroup;
  p.chunk = (int)chunk;
  p.splits = (int)((tokens + chunk - 1) / chunk);
  return p;
}

int64_t blocks_of(const KvArgs& a, const Plan& p) {
  return p.wave ? ((int64_t)a.total_tokens + 3) / 4 * a.kv_heads
                : (int64_t)a.total_tokens * a.kv_heads * p.tiles * p.splits;
}

template <int D>
hipError_t launch_d(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t, const int32_t* chosen,
                    int count, hipStream_t s) {
  const Plan p = plan(a, t.q_heads, count);
  const int64_t blocks = blocks_of(a, p);
  if (blocks > max_grid(kBlockThreads)) return hipErrorInvalidValue;
  if (p.wave) {
    auto* const kernel = p.group <= 4 ? k_kv_attn_pages_wave<D, 4> : k_kv_attn_pages_wave<D, 2>;
    kernel<<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, r, t, chosen, count, p.group);
    return hipGetLastError();
  }
  k_kv_attn_pages<D><<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, r, t, chosen, count, p.group, p.tiles,
                                                                p.splits, p.chunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (of few rows a block each is faster from five splits on: 32 rows of 8 splits 11.6 us
  // and 10.4, of 16 14.7 and 10.9, 512 of 16 13.3 and 11.9, 1024 of 8 21.9 and 22.0)
  const int64_t rows = (int64_t)a.total_tokens * t.q_heads;
  return launch_join<D>(t.part, rows, p.splits, t.out, s, rows < 1024 ? 4 : kFewSplits);
}

}  // namespace

bool attn_pages_fits(const KvArgs& a, int q_heads, int count) {
  return blocks_of(a, plan(a, q_heads, count)) <= max_grid(kBlockThreads);
}

size_t attn_pages_workspace_bytes(const KvArgs& a, int q_heads, int count) {
  const Plan p = plan(a, q_heads, count);
  if (p.splits <= 1) return 0;
  return (size_t)a.total_tokens * q_heads * (p.splits * ((int64_t)a.head_dim + 2) + 1) * sizeof(float);
}

hipError_t launch_kv_attention_pages(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t,
                                     const int32_t* chosen, int count, hipStream_t s) {
  switch (a.head_dim) {
    case 64: return launch_d<64>(a, r, t, chosen, count, s);
    case 80: return launch_d<80>(a, r, t, chosen, count, s);
    case 96: return launch_d<96>(a, r, t, chosen, count, s);
    case 128: return launch_d<128>(a, r, t, chosen, count, s);
    default: return launch_d<256>(a, r, t, chosen, count, s);
  }
}

}  // namespace i8mm
