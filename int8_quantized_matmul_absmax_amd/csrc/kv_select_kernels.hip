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

// Mean keys: one wave a page and head. Lane (t, c) of 16 x 4 takes token t of each
// block and the 16 features of tiles c, c + 4, ...; sums are 64-bit, a code's product
// with its block's 32-bit step exact in them.
template <int D>
__global__ __launch_bounds__(kBlockThreads) void k_kv_page_means(KvArgs a, uint16_t* means, int tasks) {
  const int lane = threadIdx.x & 63;
  const int task = blockIdx.x * (kBlockThreads / kWave) +
                   __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= tasks) return;
  const int b = blockIdx.y, h = task % a.kv_heads;
  const KvSeq sq = kv_seq(a, b);
  if (sq.n <= 0) return;
  const int page_tokens = a.slots * kKvBlock;
  const int j = max(sq.first, 0) / page_tokens + task / a.kv_heads;
  const int held = min(sq.len - j * page_tokens, page_tokens);
  if (held <= 0) return;
  const int page = a.page_table[(int64_t)b * a.max_pages + j];
  if ((uint32_t)page >= (uint32_t)a.num_pages) return;
  const int64_t head = (int64_t)page * a.kv_heads + h;
  const int blocks = (held + kKvBlock - 1) / kKvBlock;
  const int t = lane & 15;
  const int8_t* const codes = a.k_codes + head * a.slots * (kKvBlock * D);
  const float* const absmax = a.k_absmax + head * a.slots;
  for (int c = lane >> 4; c < (D / 16 + 3) / 4 * 4; c += 4) {
    const bool here = c < D / 16;
    double sum[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = 0.0;
    for (int s = 0; s < blocks; ++s) {
      const double step = (double)(absmax[s] / 127.0f);
      v4i32 w = {0, 0, 0, 0};
      if (here) w = ld16v(codes + (int64_t)s * (kKvBlock * D) + c * kTile + t * 16);
      if (s * kKvBlock + t >= held) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        sum[e] += step * (double)(int8_t)((uint32_t)w[e >> 2] >> (8 * (e & 3)));
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sum[e] += __shfl_xor(sum[e], d, kWave);
    }
    if (here && t == 0) {
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = f2h2((float)(sum[2 * e] / held), (float)(sum[2 * e + 1] / held));
      uint16_t* const dst = means + head * D + 16 * c;
      *reinterpret_cast<v4i32*>(dst) = v4i32{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
      *reinterpret_cast<v4i32*>(dst + 8) = v4i32{(int)o[4], (int)o[5], (int)o[6], (int)o[7]};
    }
  }
}

// The order of doubles as integers, NaN as -infinity: 0x000f... for that.
__device__ __forceinline__ uint64_t score_key(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  if ((b << 1) > (0x7ffull << 53)) return 0x000fffffffffffffull;
  return b ^ ((uint64_t)((int64_t)b >> 63) | (1ull << 63));
}

// One block a token and head. Keys of all candidate pages stand in LDS; the least of
// the chosen is found digit by digit, from histograms of 256.
template <int D, int kThreads>
__global__ __launch_bounds__(kThreads) void k_kv_select_pages(KvArgs a, RotaryArgs rot,
                                                              const uint16_t* q, int64_t q_ts,
                                                              int64_t q_hs, int group,
                                                              const uint16_t* means, int count,
                                                              int first, int recent, int32_t* out) {
  constexpr int kWaves = kThreads / kWave;
  constexpr int kLanes = D == 64 ? 8 : D <= 128 ? 16 : 32;   // of a page
  extern __shared__ uint64_t s_key[];
  __shared__ double s_sum[D], s_q[D];
  __shared__ int s_hist[256], s_wave[kWaves], s_pick[2];
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

  // the sum of the head's queries, rotated
  for (int d = tid; d < D; d += kThreads) {
    double x = 0.0;
    const uint16_t* row = q + (int64_t)token * q_ts + (int64_t)h * group * q_hs + d;
    for (int g = 0; g < group; ++g) x += (double)h2f(row[g * q_hs]);
    s_sum[d] = x;
  }
  __syncthreads();
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
  __syncthreads();

  // keys of the pages first .. seen - recent - 1
  const int candidates = seen - first - recent, want = count - first - recent;
  const int part = lane % kLanes;
  double qd[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) qd[e] = 8 * part + e < D ? s_q[8 * part + e] : 0.0;
  for (int c0 = tid / kLanes; c0 < candidates; c0 += kThreads / kLanes) {
    const int page = a.page_table[(int64_t)b * a.max_pages + first + c0];
    double s = 0.0;
    if ((uint32_t)page < (uint32_t)a.num_pages && 8 * part < D) {
      const v4i32 w = ld16v(means + ((int64_t)page * a.kv_heads + h) * D + 8 * part);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        s = __builtin_fma(qd[e], (double)h2f(((uint32_t)w[e >> 1] >> (16 * (e & 1))) & 0xffffu), s);
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) s += __shfl_xor(s, d, kWave);
    if (part == 0)
      s_key[c0] = (uint32_t)page < (uint32_t)a.num_pages ? score_key(s) : score_key(__builtin_nan(""));
  }
  __syncthreads();

  // the key of place `want`, and how many of its equals are chosen
  uint64_t least = want > 0 ? 0 : ~0ull;
  int left = want;
  for (int shift = 56; shift >= 0 && want > 0; shift -= 8) {
    for (int x = tid; x < 256; x += kThreads) s_hist[x] = 0;
    __syncthreads();
    for (int c = tid; c < candidates; c += kThreads) {
      const uint64_t k = s_key[c];
      if (shift == 56 || (k >> (shift + 8)) == (least >> (shift + 8)))
        atomicAdd(&s_hist[(int)(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < kWave) {
      // digits from the highest down, four a lane
      int n[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        n[e] = s_hist[255 - (4 * lane + e)];
        sum += n[e];
      }
      int before = wave_inclusive_scan_dpp(sum) - sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < left && left <= before + n[e]) {
          s_pick[0] = 255 - (4 * lane + e);
          s_pick[1] = left - before;
        }
        before += n[e];
      }
    }
    __syncthreads();
    least |= (uint64_t)s_pick[0] << shift;
    left = s_pick[1];
  }

  // the chosen in ascending order: the first, the best, the newest
  for (int j = tid; j < first; j += kThreads) line[j] = j;
  for (int j = tid; j < recent; j += kThreads) line[count - recent + j] = seen - recent + j;
  int placed = first, equals = 0;
  for (int c0 = 0; c0 < candidates; c0 += kThreads) {
    const int c = c0 + tid;
    const uint64_t k = c < candidates ? s_key[c] : 0;
    const bool equal = c < candidates && k == least;
    int total;
    const int rank = equals + block_prefix<kWaves>(equal, s_wave, &total);
    equals += total;
    const bool take = c < candidates && (k > least || (equal && rank < left));
    const int at = placed + block_prefix<kWaves>(take, s_wave, &total);
    placed += total;
    if (take) line[at] = first + c;
  }
}

}  // namespace

hipError_t launch_kv_page_means(const KvArgs& a, uint16_t* means, hipStream_t s) {
  const int64_t page_tokens = (int64_t)a.slots * kKvBlock;
  // pages that the new tokens of one sequence can touch
  const int64_t pages = std::min<int64_t>((a.max_tokens + 2 * page_tokens - 2) / page_tokens, a.max_pages);
  const int64_t tasks = pages * a.kv_heads;
  if (tasks > INT32_MAX - 4) return hipErrorInvalidValue;
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
#define CALL_T(D, T)                                                                             \
  do {                                                                                           \
    if (blocks > UINT32_MAX / T) return hipErrorInvalidValue;                                    \
    k_kv_select_pages<D, T><<<(uint32_t)blocks, T, lds, s>>>(a, r, q, q_ts, q_hs, group, means,  \
                                                             count, first, recent, out);         \
  } while (0)
#define CALL(D) \
  if (candidates > 512) CALL_T(D, 1024); else CALL_T(D, 256)
  I8MM_KV_DIMS(a.head_dim, CALL)
#undef CALL
#undef CALL_T
  return hipGetLastError();
}

}  // namespace i8mm
