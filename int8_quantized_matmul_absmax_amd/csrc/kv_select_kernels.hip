// The choice of the pages that a query attends to: the mean key of each page, and
// the pages whose means score best.
//
// A page's score for a token and a key/value head is the sum, over the query heads
// that share the head, of the rotated query's product with the page's mean key. Scores
// of two pages may be close, and which of them is chosen should not depend on the
// order of a sum: scores are 64-bit, from the queries' and means' 16 bits on.

#include <algorithm>

#include "kv_common.h"

namespace i8mm {

namespace {

// A double of another lane by a DPP move.
template <int kControl>
__device__ __forceinline__ double dpp_double(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kControl, 0xf, 0xf, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kControl, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The sum over 16 neighbouring lanes, in each of them: within quads (quad_perm), then
// with the mirror image in eight lanes and in sixteen.
__device__ __forceinline__ double sum_of_lanes(double x) {
  x += dpp_double<0xb1>(x);
  x += dpp_double<0x4e>(x);
  x += dpp_double<0x141>(x);
  x += dpp_double<0x140>(x);
  return x;
}
// Of kN (8 or 16) values in each of kN lanes, lane i gets the sum of the i-th: halves
// are exchanged with the mirror image, of which a lane keeps the half that its own
// number is in. 15 additions for 16 sums, by sum_of_lanes they would be 64.
template <int kControl, int kN>
__device__ __forceinline__ void exchange_halves(double* x, bool upper) {
#pragma unroll
  for (int k = 0; k < kN / 2; ++k) {
    const double keep = upper ? x[k + kN / 2] : x[k], give = upper ? x[k] : x[k + kN / 2];
    x[k] = keep + dpp_double<kControl>(give);
  }
}
template <int kN>
__device__ __forceinline__ double spread_sums(double* x, int lane) {
  if constexpr (kN == 16) exchange_halves<0x140, 16>(x, lane & 8);   // lane ^ 15
  exchange_halves<0x141, 8>(x, lane & 4);                            // lane ^ 7
  exchange_halves<0x1b, 4>(x, lane & 2);                             // lane ^ 3
  exchange_halves<0xb1, 2>(x, lane & 1);                             // lane ^ 1
  return x[0];
}

// Mean keys: one wave a page, head and 64 features (four tiles). Lane (t, c) of 16 x 4
// takes token t of each block and the 16 features of its tile; sums are 64-bit, a code's
// product with its block's 32-bit step exact in them. Eight blocks are loaded at once:
// with few pages to do, what counts is how often a wave waits (one page of 128 tokens of 8
// heads of 128 features 5.5 us, 64 pages of 16 5.2).
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_page_means(KvArgs a, uint16_t* means, int tasks) {
  constexpr int kParts = (D + 63) / 64, kBlocks = 8;
  const int lane = threadIdx.x & 63;
  const int task = blockIdx.x * (kBlockThreads / kWave) +
                   __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= tasks) return;
  const int b = blockIdx.y, part = task % kParts, h = task / kParts % a.kv_heads;
  const KvSeq sq = kv_seq(a, b);
  if (sq.n <= 0) return;
  const int page_tokens = a.slots * kKvBlock;
  const int j = max(sq.first, 0) / page_tokens + task / kParts / a.kv_heads;
  const int held = min(sq.len - j * page_tokens, page_tokens);
  if (held <= 0) return;
  const int page = a.page_table[(int64_t)b * a.max_pages + j];
  if ((uint32_t)page >= (uint32_t)a.num_pages) return;
  const int64_t head = (int64_t)page * a.kv_heads + h;
  const int blocks = (held + kKvBlock - 1) / kKvBlock;
  const int t = lane & 15, c = 4 * part + (lane >> 4);
  const bool here = c < D / 16;
  const int8_t* const codes =
      a.k_codes + head * a.slots * (kKvBlock * D) + min(c, D / 16 - 1) * kTile + t * 16;
  const float* const absmax = a.k_absmax + head * a.slots;
  double sum[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[e] = 0.0;
  for (int s0 = 0; s0 < blocks; s0 += kBlocks) {
    v4i32 w[kBlocks];
    float a_block[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int s = min(s0 + u, blocks - 1);
      a_block[u] = absmax[s];
      w[u] = ld16v(codes + (int64_t)s * (kKvBlock * D));
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      if (s0 + u >= blocks) continue;
      // (a token past the end may hold anything in a block that counts)
      const double step = (s0 + u) * kKvBlock + t < held ? (double)(a_block[u] / 127.0f) : 0.0;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        sum[e] += step * (double)(int8_t)((uint32_t)w[u][e >> 2] >> (8 * (e & 3)));
    }
  }
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[e] = sum_of_lanes(sum[e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = f2h2((float)(sum[2 * e] / held), (float)(sum[2 * e + 1] / held));
  if (here && t == 0) {
    uint16_t* const dst = means + head * D + 16 * c;
    *reinterpret_cast<v4i32*>(dst) = v4i32{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
    *reinterpret_cast<v4i32*>(dst + 8) = v4i32{(int)o[4], (int)o[5], (int)o[6], (int)o[7]};
  }
}

// The order of doubles as integers, NaN as -infinity, which is kNoScore.
constexpr uint64_t kNoScore = 0x000fffffffffffffull;
__device__ __forceinline__ uint64_t score_key(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  if ((b << 1) > (0x7ffull << 53)) return kNoScore;
  return b ^ ((uint64_t)((int64_t)b >> 63) | (1ull << 63));
}

// One block a token and head. Keys of all candidate pages stand in LDS; the least of
// the chosen is found digit by digit, from histograms of 256.
//
// A page's mean is taken by kLanes lanes, eight features each. What a block waits for
// is kept to a few times: a group of lanes loads as many entries of the page table at
// once, then the means of kAhead pages; kBatch pages' sums are made together. One token
// over 1024 pages, 8 heads of 128 features: 12.9 us, of which the scores 6 (64-bit sums
// of eight blocks) and the rest waits; 64 tokens over up to 512 pages 15.1.
template <int D, int kThreads>
__global__ __launch_bounds__(kThreads) void k_kv_select_pages(KvArgs a, RotaryArgs rot,
                                                              const uint16_t* q, int64_t q_ts,
                                                              int64_t q_hs, int group,
                                                              const uint16_t* means, int count,
                                                              int first, int recent, int32_t* out) {
  constexpr int kWaves = kThreads / kWave;
  constexpr int kLanes = D == 64 ? 8 : D <= 128 ? 16 : 32;   // of a page
  constexpr int kGroups = kThreads / kLanes, kBatch = kLanes < 16 ? kLanes : 16, kAhead = 8;
  extern __shared__ uint64_t s_key[];
  __shared__ double s_sum[D], s_q[D];
  __shared__ int s_hist[3][256], s_wave[kWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int token = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
  const int b = sequence_of(a, token, lane);
  const KvSeq sq = kv_seq(a, b);
  const int i = token - sq.row0, pos = sq.first + i;
  const int page_tokens = a.slots * kKvBlock;
  const int seen = i >= 0 && i < sq.n && pos >= 0 ? pos / page_tokens + 1 : 0;
  int32_t* const line = out + (int64_t)blockIdx.x * count;
  if (seen <= count) {
    for (int j = tid; j < count; j += kThreads) line[j] = j < seen ? j : -1;
    return;
  }
  const int candidates = seen - first - recent, want = count - first - recent;
  for (int j = tid; j < first; j += kThreads) line[j] = j;
  for (int j = tid; j < recent; j += kThreads) line[count - recent + j] = seen - recent + j;

  // the sum of the head's queries, rotated
  for (int d = tid; d < D; d += kThreads) {
    const uint16_t* const row = q + (int64_t)token * q_ts + (int64_t)h * group * q_hs + d;
    double x = 0.0;
    for (int g0 = 0; g0 < group; g0 += 8) {
      uint32_t v[8];
#pragma unroll
      for (int g = 0; g < 8; ++g) v[g] = row[min(g0 + g, group - 1) * q_hs];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g0 + g < group) x += (double)h2f(v[g]);
    }
    s_sum[d] = x;
  }
  for (int x = tid; x < 256; x += kThreads) s_hist[0][x] = 0;
  lds_only_barrier();
  for (int d = tid; d < D; d += kThreads) {
    double x = s_sum[d];
    if (rot.cos && d < rot.dim) {
      const int half = rot.dim >> 1;
      const int k = rot.interleaved ? d >> 1 : d < half ? d : d - half;
      const bool low = rot.interleaved ? !(d & 1) : d < half;
      const int o = rot.interleaved ? d ^ 1 : low ? d + half : d - half;
      const int64_t at = (int64_t)pos * half + k;
      const double own = x * (double)rot.cos[at], far = s_sum[o] * (double)rot.sin[at];
      x = low ? own - far : own + far;
    }
    s_q[d] = x;
  }
  lds_only_barrier();

  // keys of the pages first .. seen - recent - 1
  const int part = tid % kLanes, mine = tid / kLanes;
  const bool here = 8 * part < D;
  double qd[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) qd[e] = here ? s_q[8 * part + e] : 0.0;
  const int32_t* const entries = a.page_table + (int64_t)b * a.max_pages + first;
  for (int c0 = 0; c0 < candidates; c0 += kThreads) {
    const int c = c0 + part * kGroups + mine;
    const int entry = c < candidates ? page_or_none(a, entries[c]) : -1;
#pragma unroll 1
    for (int k0 = 0; k0 < kLanes && c0 + k0 * kGroups < candidates; k0 += kBatch) {
      double s[kBatch];
#pragma unroll
      for (int u0 = 0; u0 < kBatch; u0 += kAhead) {
        v4i32 w[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int page = __shfl(entry, (lane - part) + k0 + u0 + u, kWave);
          w[u] = v4i32{0, 0, 0, 0};
          if (here && page >= 0) w[u] = ld16v(means + ((int64_t)page * a.kv_heads + h) * D + 8 * part);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          s[u0 + u] = 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            s[u0 + u] = __builtin_fma(
                qd[e], (double)h2f(((uint32_t)w[u][e >> 1] >> (16 * (e & 1))) & 0xffffu), s[u0 + u]);
        }
      }
      // (each lane now gets the score of its own entry)
      double mine_sum = spread_sums<kBatch>(s, lane);
      if constexpr (kLanes == 32) mine_sum += __shfl_xor(mine_sum, 16, kWave);
      if (part / kBatch == k0 / kBatch && c < candidates)
        s_key[c] = entry >= 0 ? score_key(mine_sum) : kNoScore;
    }
  }
  lds_only_barrier();

  // the key of place `want`, and how many of its equals are chosen. (Every wave reads
  // the histogram for itself; the next one is cleared two barriers before it is read.)
  uint64_t least = want > 0 ? 0 : ~0ull;
  int left = want;
  for (int digit = 0; digit < 8 && want > 0; ++digit) {
    const int shift = 56 - 8 * digit;
    int* const hist = s_hist[digit % 3];
    for (int x = tid; x < 256; x += kThreads) s_hist[(digit + 1) % 3][x] = 0;
    for (int c = tid; c < candidates; c += kThreads) {
      const uint64_t k = s_key[c];
      if (digit == 0 || (k >> (shift + 8)) == (least >> (shift + 8)))
        atomicAdd(&hist[(int)(k >> shift) & 255], 1);
    }
    lds_only_barrier();
    // digits from the highest down, four a lane
    int n[4], sum = 0, pick = -1, rest = 0, many = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[e] = hist[255 - (4 * lane + e)];
      sum += n[e];
    }
    int before = wave_inclusive_scan_dpp(sum) - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (before < left && left <= before + n[e]) {
        pick = 255 - (4 * lane + e);
        rest = left - before;
        many = n[e];
      }
      before += n[e];
    }
    const int from = __builtin_ctzll(__ballot(pick >= 0));
    least |= (uint64_t)__builtin_amdgcn_readlane(pick, from) << shift;
    left = __builtin_amdgcn_readlane(rest, from);
    if (left == __builtin_amdgcn_readlane(many, from)) break;   // all that begin with these digits
  }

  // The chosen in ascending order between the first and the newest. A page's place:
  // those above the least before it, and of those that are equal at most `left`. (After
  // an early end none is equal but by chance, and then all are chosen.)
  int placed = 0;   // above the least, and equals in the upper half
  for (int c0 = 0; c0 < candidates; c0 += kThreads) {
    const int c = c0 + tid;
    const uint64_t k = c < candidates ? s_key[c] : 0;
    const int above = c < candidates && k > least, equal = c < candidates && k == least;
    int total;
    const int at = placed + block_prefix<kWaves>(above | equal << 16, s_wave, &total);
    placed += total;
    const int equals = at >> 16;
    if (above || (equal && equals < left)) line[first + (at & 0xffff) + min(equals, left)] = first + c;
  }
}

}  // namespace

int64_t page_means_tasks(const KvArgs& a) {
  const int64_t page_tokens = (int64_t)a.slots * kKvBlock;
  // pages that the new tokens of one sequence can touch
  const int64_t pages = std::min<int64_t>((a.max_tokens + 2 * page_tokens - 2) / page_tokens, a.max_pages);
  return pages * a.kv_heads * ((a.head_dim + 63) / 64);
}

hipError_t launch_kv_page_means(const KvArgs& a, uint16_t* means, hipStream_t s) {
  const int64_t tasks = page_means_tasks(a);
  if ((tasks + 3) / 4 > max_grid(kBlockThreads)) return hipErrorInvalidValue;
  if (tasks == 0) return hipSuccess;
  const dim3 grid((uint32_t)((tasks + 3) / 4), (uint32_t)a.num_seqs);
#define CALL(D) k_kv_page_means<D><<<grid, kBlockThreads, 0, s>>>(a, means, (int)tasks)
  I8MM_KV_DIMS(a.head_dim, CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t launch_kv_select_pages(const KvArgs& a, const RotaryArgs& r, const uint16_t* q, int64_t q_ts,
                                  int64_t q_hs, int q_heads, const uint16_t* means, int count, int first,
                                  int recent, int32_t* out, hipStream_t s) {
  const int64_t blocks = (int64_t)a.total_tokens * a.kv_heads;
  const int64_t pages = ((int64_t)a.len_cap + a.slots * kKvBlock - 1) / (a.slots * kKvBlock);
  const int64_t candidates = std::max<int64_t>(pages - first - recent, 0);
  if (candidates > kMaxSelectPages) return hipErrorInvalidValue;
  const int group = q_heads / a.kv_heads;
  const size_t lds = (size_t)candidates * 8;
#define CALL_T(D, T)                                                                            \
  k_kv_select_pages<D, T><<<(uint32_t)blocks, T, lds, s>>>(a, r, q, q_ts, q_hs, group, means,   \
                                                           count, first, recent, out)
  const int threads = select_threads(blocks, candidates);
  if (blocks > max_grid(threads)) return hipErrorInvalidValue;
#define CALL(D) \
  if (threads == 1024) CALL_T(D, 1024); else CALL_T(D, 256)
  I8MM_KV_DIMS(a.head_dim, CALL)
#undef CALL
#undef CALL_T
  return hipGetLastError();
}

}  // namespace i8mm
