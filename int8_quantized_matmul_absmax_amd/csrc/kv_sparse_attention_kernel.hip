// Attention over chosen pages of the paged 8-bit key/value cache.
//
// Each token and key/value head has its own list of pages, so its rows are only the
// query heads that share the head: a block takes up to 16 of them, its waves stream
// the pages' blocks through LDS as the dense kernel for few rows does, with the same
// arithmetic. A list's tokens are counted on from page to page: groups of 64 of them
// may begin inside one page and end in another.

#include "kv_attention_common.h"

namespace i8mm {

namespace {

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

  // entries of the list up to the last page that may be visible
  const int32_t* const list = chosen + ((int64_t)token * a.kv_heads + h) * count;
  const int page_tokens = a.slots * kKvBlock;
  const int seen_pages = belongs ? pos / page_tokens + 1 : 0;
  int entries = 0;
  for (int e0 = 0; e0 < count; e0 += kWave) {
    const int e = e0 + lane;
    const uint64_t there = __ballot(e < count && (uint32_t)list[min(e, count - 1)] < (uint32_t)seen_pages);
    if (there) entries = e0 + 64 - __builtin_clzll(there);
  }
  const int all = entries * page_tokens;
  const int begin = split * chunk, end = min(begin + chunk, all);
  const bool only = all <= chunk;
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
    if (splits > 1 && split == 0 && d4 == 0) parts.count[out_row] = (all + chunk - 1) / chunk;
  }
}

// Splits of a list's tokens, as for few rows of the dense attention.
struct Plan {
  int group, tiles, splits, chunk;
};
Plan plan(const KvArgs& a, int q_heads, int count) {
  constexpr int64_t kMinChunk = 4 * kGroup, kMaxChunk = 2048, kMaxSplits = 1024;
  const int64_t resident = (a.head_dim <= 128 ? 2 : 1) * 256;
  Plan p;
  p.group = q_heads / a.kv_heads;
  p.tiles = (p.group + kRows - 1) / kRows;
  const int64_t tokens = (int64_t)count * a.slots * kKvBlock;
  const int64_t blocks = (int64_t)a.total_tokens * a.kv_heads * p.tiles;
  int64_t chunk = std::min<int64_t>(std::max(tokens * blocks / resident, kMinChunk), kMaxChunk);
  chunk = std::max(chunk, tokens / kMaxSplits + 1);
  chunk = (chunk + kGroup - 1) / kGroup * kGroup;
  p.chunk = (int)chunk;
  p.splits = (int)((tokens + chunk - 1) / chunk);
  return p;
}

template <int D>
hipError_t launch_d(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t, const int32_t* chosen,
                    int count, hipStream_t s) {
  const Plan p = plan(a, t.q_heads, count);
  const int64_t blocks = (int64_t)a.total_tokens * a.kv_heads * p.tiles * p.splits;
  if (blocks > UINT32_MAX / kBlockThreads) return hipErrorInvalidValue;
  k_kv_attn_pages<D><<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, r, t, chosen, count, p.group, p.tiles,
                                                                p.splits, p.chunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_join<D>(t.part, (int64_t)a.total_tokens * t.q_heads, p.splits, t.out, s);
}

}  // namespace

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
