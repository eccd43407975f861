// Pages of the paged key/value cache: the step of the page tables between two
// appends, compaction, and the copies that either asks for.
//
// No state is kept between calls: a page is free when no row of the new table
// names it, so each call marks the pages that are named, in a word for each page,
// and one block then gives out free ones in ascending order. What the tables hold
// is bounded on the device, as the cache's calls do.

#include <algorithm>

#include "kv_common.h"

namespace i8mm {

namespace {

constexpr int kOneBlock = 1024;   // threads of the block that gives out pages
constexpr int kOneWaves = kOneBlock / kWave;

// A page's word: 0, or of the references to it the greatest: kRead for a row that
// will not write to the page, rows - i for row i that will. So a page that some row
// only reads is copied by all that write to it, and otherwise by all but the first.
constexpr uint32_t kRead = 0xffffffffu;

// Calls up to these sizes are one block's work in one launch: the words, the free
// pages and the rows stand in its LDS. Larger ones mark pages with a grid and give them
// out with a block after it. A step of 4 rows of 17 entries 4.4 us against 7.7, 64 of
// 128 7.1 and 10.9, 256 of 64 10.3 and 13.0, 256 of 131 14.5 and 11.7, 512 of 128 24.9
// and 18.2; a compaction 5.6 and 9.6, 7.0 and 11.4, 11.9 and 16.8, 16.9 and 11.6, 32 and
// 25. That is recorded; an eager launch saved is 2 to 3 us of the host's, and 256 rows
// of 131 with their copies in two layers 27.7 us against 30.9.
constexpr int kOneRows = 1024, kOnePages = 16384, kOneEntries = 40960;

// What row i of a step takes of its parent.
struct Row {
  int parent;      // or -1
  int pages;       // of the tokens kept
  int all_pages;
  int rest;        // tokens kept in the last of `pages`, 0 if they fill it
  bool writes;     // to that page
  bool full;       // not all of its new tokens have room
};
// (*batch_len: its length in a batch of the new tokens)
__device__ __forceinline__ Row step_row(const PagesArgs& a, int i, int* len, int* batch_len) {
  const int limit = min(a.max_pages * a.page_tokens, a.max_len);
  Row r;
  r.parent = a.parents[i];
  if ((uint32_t)r.parent >= (uint32_t)a.num_seqs) r.parent = -1;
  const int keep = a.keep ? max(a.keep[i], 0) : limit;
  const int more = max(a.new_tokens ? a.new_tokens[i] : a.new_all, 0);
  int kept = r.parent >= 0 ? min(max(a.seq_lens[r.parent], 0), limit) : 0;
  kept = min(kept, keep);
  *len = kept + min(more, limit - kept);
  r.pages = (kept + a.page_tokens - 1) / a.page_tokens;
  r.all_pages = (*len + a.page_tokens - 1) / a.page_tokens;
  r.rest = kept - kept / a.page_tokens * a.page_tokens;
  r.writes = r.rest != 0 && *len > kept;
  r.full = more > limit - kept;
  *batch_len = more > 0 && !r.full ? *len : 0;
  return r;
}
__device__ __forceinline__ int4 packed(const Row& r) {
  return make_int4(r.parent, r.pages, r.all_pages,
                   r.rest | (r.writes ? 1 << 30 : 0) | (r.full ? 1 << 29 : 0));
}
__device__ __forceinline__ Row unpacked(const int4& p) {
  return Row{p.x, p.y, p.z, p.w & 0xffff, (p.w & 1 << 30) != 0, (p.w & 1 << 29) != 0};
}

__device__ __forceinline__ int page_or_none(const PagesArgs& a, int page) {
  return (uint32_t)page < (uint32_t)a.num_pages ? page : -1;
}

// Entries of a row that its parent's tokens keep, and what they say of the pages.
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_keep(PagesArgs a, uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  if (j >= a.max_pages) return;
  int len, batch_len;
  const Row r = step_row(a, i, &len, &batch_len);
  int page = -1;
  if (j < r.pages) page = page_or_none(a, a.page_table[(int64_t)r.parent * a.max_pages + j]);
  a.out_table[(int64_t)i * a.max_pages + j] = page;
  if (page < 0) return;
  if (r.writes && j == r.pages - 1)
    __hip_atomic_fetch_max(words + page, (uint32_t)(a.num_rows - i), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
  else
    __hip_atomic_store(words + page, kRead, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The first `want` pages whose word is 0, to list; how many there are of them.
__device__ __forceinline__ int list_free(const uint32_t* words, int num_pages, int want,
                                         int32_t* list, int* s_wave) {
  constexpr int kEach = 8;
  int found = 0;
  for (int p0 = 0; p0 < num_pages && found < want; p0 += kEach * kOneBlock) {
    const int p = p0 + kEach * (int)threadIdx.x;
    uint32_t w[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) w[e] = p + e < num_pages ? words[p + e] : 1u;
    int n = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) n += w[e] == 0;
    int total;
    int at = found + block_prefix<kOneWaves>(n, s_wave, &total);
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (w[e] == 0) {
        if (at < want) list[at] = p + e;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// New pages of all rows, in their order: of each first the copy of the page that it
// shares and will write to, then those of tokens that begin a page. One block;
// row_of(i) is row i.
template <class RowOf>
__device__ __forceinline__ void give_pages(const PagesArgs& a, const uint32_t* words, int32_t* list,
                                           int2* places, int* s_wave, RowOf row_of) {
  const int tid = threadIdx.x, lane = tid & 63;
  int want = 0, copies = 0, full = 0;
  for (int i0 = 0; i0 < a.num_rows; i0 += kOneBlock) {
    const int i = i0 + tid;
    int copy = 0, need = 0, no_room = 0;
    if (i < a.num_rows) {
      const Row r = row_of(i);
      no_room = r.full;
      if (r.writes) {
        const int page = a.out_table[(int64_t)i * a.max_pages + r.pages - 1];
        copy = page >= 0 && words[page] != (uint32_t)(a.num_rows - i);
      }
      need = copy + r.all_pages - r.pages;
    }
    int total;
    const int at = want + block_prefix<kOneWaves>(need, s_wave, &total);
    want += total;
    // (both counts are a block's threads at most)
    const int rank = copies + (block_prefix<kOneWaves>(copy | no_room << 16, s_wave, &total) & 0xffff);
    copies += total & 0xffff;
    full += total >> 16;
    if (i < a.num_rows) places[i] = int2{at, copy ? rank : -1};
  }
  const int have = list_free(words, a.num_pages, want, list, s_wave);
  int done = 0;
  for (int i0 = 0; i0 < a.num_rows; i0 += kOneBlock) {
    const int i = i0 + tid;
    int made = 0, at = 0, extra = 0, first = 0;
    if (i < a.num_rows) {
      const Row r = row_of(i);
      const int2 place = places[i];
      int32_t* const row = a.out_table + (int64_t)i * a.max_pages;
      at = place.x;
      if (place.y >= 0) {
        const int from = row[r.pages - 1], to = at < have ? list[at] : -1;
        row[r.pages - 1] = to;
        ++at;
        if (to >= 0) {
          int32_t* const c = a.copies + 3 * (int64_t)place.y;
          c[0] = from;
          c[1] = to;
          c[2] = r.rest;
          made = 1;
        }
      }
      first = r.pages;
      extra = r.all_pages - r.pages;
      if (extra > 0) row[first] = at < have ? list[at] : -1;
    }
    // Rows with more new pages than one: by a thread each, or each in turn by a wave's
    // lanes. A turn takes the time of four pages of a thread: 190 rows of 6 pages 18.2 us
    // in turn and 9.3 by their threads, 64 of 42 18.7 and 11.4.
    const int few = 4 * __popcll(__ballot(extra > 1));
    if (extra > 1 && extra <= few) {
      int32_t* const row = a.out_table + (int64_t)i * a.max_pages + first;
#pragma unroll 4
      for (int j = 1; j < extra; ++j) row[j] = at + j < have ? list[at + j] : -1;
    }
    uint64_t long_rows = __ballot(extra > few && extra > 1);
    while (long_rows) {
      const int from = __builtin_ctzll(long_rows);
      long_rows &= long_rows - 1;
      const int n = __builtin_amdgcn_readlane(extra, from), l0 = __builtin_amdgcn_readlane(at, from);
      const int j0 = __builtin_amdgcn_readlane(first, from);
      int32_t* const row = a.out_table + (int64_t)(i0 + (tid & ~63) + from) * a.max_pages + j0;
      for (int j = 1 + lane; j < n; j += kWave) row[j] = l0 + j < have ? list[l0 + j] : -1;
    }
    int total;
    block_prefix<kOneWaves>(made, s_wave, &total);
    done += total;
  }
  // (copies are made in the order of the rows until the pages run out)
  for (int i = done + tid; i < a.num_rows; i += kOneBlock) {
    int32_t* const c = a.copies + 3 * (int64_t)i;
    c[0] = c[1] = c[2] = -1;
  }
  if (tid == 0) {
    a.counts[0] = done;
    a.counts[1] = want - have;
    if (a.full) a.full[0] = full;
  }
}

__global__ __launch_bounds__(kOneBlock) void k_kv_pages_give(PagesArgs a, const uint32_t* words,
                                                             int32_t* list, int2* places) {
  __shared__ int s_wave[kOneWaves];
  for (int i = threadIdx.x; i < a.num_rows; i += kOneBlock) {
    int len, batch_len;
    step_row(a, i, &len, &batch_len);
    a.out_lens[i] = len;
    if (a.batch_lens) a.batch_lens[i] = batch_len;
  }
  give_pages(a, words, list, places, s_wave, [&](int i) {
    int len, batch_len;
    return step_row(a, i, &len, &batch_len);
  });
}

// A thread's entries of a table, kOneBlock apart: entry j of row i. (A division for
// each costs more than the rest of its work: 34000 entries 18.5 us, so 14.4; a wave a
// row at a time 22.)
struct Entry {
  int i, j, di, dj, width;
  __device__ __forceinline__ explicit Entry(int max_pages) {
    width = max(max_pages, 1);
    i = (int)threadIdx.x / width;
    j = (int)threadIdx.x - i * width;
    di = kOneBlock / width;
    dj = kOneBlock - di * width;
  }
  __device__ __forceinline__ void next() {
    i += di;
    j += dj;
    if (j >= width) {
      j -= width;
      ++i;
    }
  }
};

// Both in one block. kAhead of a thread's entries are in flight at once (with 16 the
// same, with 32 slower: their bounds are checked where there are none, too).
constexpr int kAhead = 8;
__global__ __launch_bounds__(kOneBlock) void k_kv_pages_step_one(PagesArgs a) {
  extern __shared__ __attribute__((aligned(16))) int32_t s_all[];
  __shared__ int s_wave[kOneWaves];
  int4* const rows = reinterpret_cast<int4*>(s_all);
  int2* const places = reinterpret_cast<int2*>(rows + a.num_rows);
  uint32_t* const words = reinterpret_cast<uint32_t*>(places + a.num_rows);
  int32_t* const list = reinterpret_cast<int32_t*>(words + a.num_pages);
  const int tid = threadIdx.x;
  if (tid < a.num_rows) {
    int len, batch_len;
    rows[tid] = packed(step_row(a, tid, &len, &batch_len));
    a.out_lens[tid] = len;
    if (a.batch_lens) a.batch_lens[tid] = batch_len;
  }
  for (int p = tid; p < a.num_pages; p += kOneBlock) words[p] = 0;
  __syncthreads();
  const int entries = a.num_rows * a.max_pages;
  Entry at(a.max_pages);
  for (int e0 = 0; e0 < entries; e0 += kAhead * kOneBlock) {
    int page[kAhead];
    Entry x = at;
#pragma unroll
    for (int u = 0; u < kAhead; ++u, at.next()) {
      page[u] = -1;
      if (at.i >= a.num_rows) continue;
      const int4 r = rows[at.i];
      if (at.j < r.y) page[u] = a.page_table[r.x * a.max_pages + at.j];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u, x.next()) {
      if (x.i >= a.num_rows) continue;
      const Row r = unpacked(rows[x.i]);
      const int p = page_or_none(a, page[u]);
      a.out_table[e0 + u * kOneBlock + tid] = p;
      if (p < 0) continue;
      if (r.writes && x.j == r.pages - 1)
        atomicMax(words + p, (uint32_t)(a.num_rows - x.i));
      else
        words[p] = kRead;   // (the greatest: it stays, before or after the others)
    }
  }
  __syncthreads();
  give_pages(a, words, list, places, s_wave, [&](int i) { return unpacked(rows[i]); });
}

// Compaction: pages named by a row.
__device__ __forceinline__ int used_pages(const PagesArgs& a, int i) {
  const int len = min(max(a.seq_lens[i], 0), a.max_pages * a.page_tokens);
  return (len + a.page_tokens - 1) / a.page_tokens;
}
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_used(PagesArgs a, uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  if (j >= used_pages(a, i)) return;
  const int page = page_or_none(a, a.page_table[(int64_t)i * a.max_pages + j]);
  if (page >= 0) __hip_atomic_store(words + page, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The k-th used page at or past the number of used ones goes to the k-th free one
// below it; words become the pages' new places. One block.
__device__ __forceinline__ void plan_moves(const PagesArgs& a, uint32_t* words, int32_t* list,
                                           int* s_wave) {
  constexpr int kEach = 8;
  const int tid = threadIdx.x;
  int n = 0, live;
  for (int p = tid; p < a.num_pages; p += kOneBlock) n += words[p] != 0;
  block_prefix<kOneWaves>(n, s_wave, &live);
  list_free(words, live, live, list, s_wave);
  for (int p = tid; p < live; p += kOneBlock)
    if (words[p] != 0) words[p] = (uint32_t)p;
  int moves = 0;
  for (int p0 = live; p0 < a.num_pages; p0 += kEach * kOneBlock) {
    const int p = p0 + kEach * tid;
    uint32_t w[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) w[e] = p + e < a.num_pages ? words[p + e] : 0u;
    int some = 0, total;
#pragma unroll
    for (int e = 0; e < kEach; ++e) some += w[e] != 0;
    int rank = moves + block_prefix<kOneWaves>(some, s_wave, &total);
    moves += total;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (w[e] == 0) continue;
      const int to = list[rank];
      words[p + e] = (uint32_t)to;
      int32_t* const c = a.copies + 3 * (int64_t)rank;
      c[0] = p + e;
      c[1] = to;
      c[2] = a.page_tokens;
      ++rank;
    }
  }
  for (int i = moves + tid; i < a.num_pages / 2; i += kOneBlock) {
    int32_t* const c = a.copies + 3 * (int64_t)i;
    c[0] = c[1] = c[2] = -1;
  }
  if (tid == 0) {
    a.counts[0] = moves;
    a.counts[1] = live;
  }
}
__global__ __launch_bounds__(kOneBlock) void k_kv_pages_plan(PagesArgs a, uint32_t* words,
                                                             int32_t* list) {
  __shared__ int s_wave[kOneWaves];
  plan_moves(a, words, list, s_wave);
}
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_rename(PagesArgs a,
                                                                   const uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  if (j >= a.max_pages) return;
  const int64_t at = (int64_t)i * a.max_pages + j;
  int page = -1;
  if (j < used_pages(a, i)) page = page_or_none(a, a.page_table[at]);
  a.out_table[at] = page < 0 ? -1 : (int)words[page];
}
// All three in one block.
__global__ __launch_bounds__(kOneBlock) void k_kv_pages_compact_one(PagesArgs a) {
  extern __shared__ __attribute__((aligned(16))) int32_t s_all[];
  __shared__ int s_wave[kOneWaves];
  int32_t* const used = s_all;
  uint32_t* const words = reinterpret_cast<uint32_t*>(used + a.num_seqs);
  int32_t* const list = reinterpret_cast<int32_t*>(words + a.num_pages);
  const int tid = threadIdx.x;
  if (tid < a.num_seqs) used[tid] = used_pages(a, tid);
  for (int p = tid; p < a.num_pages; p += kOneBlock) words[p] = 0;
  __syncthreads();
  const int entries = a.num_seqs * a.max_pages;
  auto load = [&](Entry& at, int (&page)[kAhead]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u, at.next()) {
      page[u] = -1;
      if (at.i < a.num_seqs && at.j < used[at.i]) page[u] = a.page_table[at.i * a.max_pages + at.j];
    }
  };
  Entry at(a.max_pages);
  for (int e0 = 0; e0 < entries; e0 += kAhead * kOneBlock) {
    int page[kAhead];
    load(at, page);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (page_or_none(a, page[u]) >= 0) words[page[u]] = 1;
  }
  __syncthreads();
  plan_moves(a, words, list, s_wave);
  __syncthreads();
  at = Entry(a.max_pages);
  for (int e0 = 0; e0 < entries; e0 += kAhead * kOneBlock) {
    int page[kAhead];
    load(at, page);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int e = e0 + u * kOneBlock + tid;
      if (e < entries) a.out_table[e] = page_or_none(a, page[u]) >= 0 ? (int)words[page[u]] : -1;
    }
  }
}

// Copies of pages. An item is a head's keys or values of one page: its blocks stand
// one after the other. Bound by memory: 1746 pages of 64 tokens, 8 heads of 128 features
// (459 MB) 84 us, 5.4 TB/s; the copies of 256 beams 6.0 us, of 4 3.4.
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_copy(KvArgs a, uint16_t* means,
                                                                 const int32_t* copies,
                                                                 const int32_t* count, int most) {
  const int64_t items = (int64_t)min(max(*count, 0), most) * a.kv_heads * 2;
  const int64_t block_bytes = (int64_t)kKvBlock * a.head_dim;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int pair = (int)(item / (2 * a.kv_heads)), h = (int)(item / 2 % a.kv_heads);
    const bool values = item & 1;
    const int32_t* const c = copies + 3 * (int64_t)pair;
    const int from = c[0], to = c[1];
    const int blocks = (min(max(c[2], 0), a.slots * kKvBlock) + kKvBlock - 1) / kKvBlock;
    if ((uint32_t)from >= (uint32_t)a.num_pages || (uint32_t)to >= (uint32_t)a.num_pages || from == to)
      continue;
    const int64_t src = ((int64_t)from * a.kv_heads + h) * a.slots;
    const int64_t dst = ((int64_t)to * a.kv_heads + h) * a.slots;
    int8_t* const codes = values ? a.v_codes : a.k_codes;
    float* const absmax = values ? a.v_absmax : a.k_absmax;
    const v4i32* const s = reinterpret_cast<const v4i32*>(codes + src * block_bytes);
    v4i32* const d = reinterpret_cast<v4i32*>(codes + dst * block_bytes);
    const int n = (int)(blocks * block_bytes / 16);
    for (int e = threadIdx.x; e < n; e += kBlockThreads)
      __builtin_nontemporal_store(__builtin_nontemporal_load(s + e), d + e);
    for (int e = threadIdx.x; e < blocks; e += kBlockThreads) absmax[dst + e] = absmax[src + e];
    if (means && !values && blocks > 0)
      for (int e = threadIdx.x; e < a.head_dim; e += kBlockThreads)
        means[dst / a.slots * a.head_dim + e] = means[src / a.slots * a.head_dim + e];
  }
}

bool one_block(const PagesArgs& a, int rows) {
  return rows <= kOneRows && a.num_pages <= kOnePages && (int64_t)rows * a.max_pages <= kOneEntries;
}

int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

}  // namespace

// words [num_pages], list [num_pages], places [rows]
size_t kv_pages_workspace_bytes(const PagesArgs& a, int rows) {
  if (one_block(a, rows)) return 0;
  return (size_t)(2 * pad4(a.num_pages) + 2 * (int64_t)rows) * 4;
}

hipError_t launch_kv_pages_step(const PagesArgs& a, void* ws, hipStream_t s) {
  if (one_block(a, a.num_rows)) {
    const size_t lds = (size_t)a.num_rows * 24 + (size_t)a.num_pages * 8;
    k_kv_pages_step_one<<<1, kOneBlock, lds, s>>>(a);
    return hipGetLastError();
  }
  uint32_t* const words = static_cast<uint32_t*>(ws);
  int32_t* const list = static_cast<int32_t*>(ws) + pad4(a.num_pages);
  int2* const places = reinterpret_cast<int2*>(list + pad4(a.num_pages));
  hipError_t e = hipSuccess;
  if (a.num_pages > 0) e = launch_fill_u32(words, a.num_pages, 0u, s);
  if (e != hipSuccess) return e;
  if (a.max_pages > 0 && a.num_rows > 0) {
    const dim3 grid((uint32_t)((a.max_pages + kBlockThreads - 1) / kBlockThreads), (uint32_t)a.num_rows);
    k_kv_pages_keep<<<grid, kBlockThreads, 0, s>>>(a, words);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_kv_pages_give<<<1, kOneBlock, 0, s>>>(a, words, list, places);
  return hipGetLastError();
}

hipError_t launch_kv_pages_compact(const PagesArgs& a, void* ws, hipStream_t s) {
  if (one_block(a, a.num_seqs)) {
    const size_t lds = (size_t)a.num_seqs * 4 + (size_t)a.num_pages * 8;
    k_kv_pages_compact_one<<<1, kOneBlock, lds, s>>>(a);
    return hipGetLastError();
  }
  uint32_t* const words = static_cast<uint32_t*>(ws);
  int32_t* const list = static_cast<int32_t*>(ws) + pad4(a.num_pages);
  hipError_t e = hipSuccess;
  if (a.num_pages > 0) e = launch_fill_u32(words, a.num_pages, 0u, s);
  if (e != hipSuccess) return e;
  const bool some = a.max_pages > 0 && a.num_seqs > 0;
  const dim3 grid((uint32_t)((a.max_pages + kBlockThreads - 1) / kBlockThreads), (uint32_t)a.num_seqs);
  if (some) {
    k_kv_pages_used<<<grid, kBlockThreads, 0, s>>>(a, words);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_kv_pages_plan<<<1, kOneBlock, 0, s>>>(a, words, list);
  e = hipGetLastError();
  if (e != hipSuccess || !some) return e;
  k_kv_pages_rename<<<grid, kBlockThreads, 0, s>>>(a, words);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const KvArgs& a, uint16_t* means, const int32_t* copies,
                                const int32_t* count, int most, hipStream_t s) {
  const int64_t items = (int64_t)most * a.kv_heads * 2;
  const int64_t blocks = std::min<int64_t>(items, 4096);
  k_kv_pages_copy<<<(uint32_t)blocks, kBlockThreads, 0, s>>>(a, means, copies, count, most);
  return hipGetLastError();
}

}  // namespace i8mm
