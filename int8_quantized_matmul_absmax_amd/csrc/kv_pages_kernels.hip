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
// only reads is copied by all that write to it, and otherwise all but the first.
constexpr uint32_t kRead = 0xffffffffu;

// What row i of a step takes of its parent.
struct Row {
  int parent;    // or -1
  int kept;      // tokens
  int len;
  int pages;     // of the kept tokens
  int all_pages;
  bool writes;   // to the last of the kept pages
};
__device__ __forceinline__ Row step_row(const PagesArgs& a, int i) {
  const int limit = a.max_pages * a.page_tokens;
  Row r;
  r.parent = a.parents[i];
  if ((uint32_t)r.parent >= (uint32_t)a.num_seqs) r.parent = -1;
  r.kept = r.parent >= 0 ? min(max(a.seq_lens[r.parent], 0), limit) : 0;
  if (a.keep) r.kept = min(r.kept, max(a.keep[i], 0));
  const int more = max(a.new_tokens ? a.new_tokens[i] : a.new_all, 0);
  r.len = r.kept + min(more, limit - r.kept);
  r.pages = (r.kept + a.page_tokens - 1) / a.page_tokens;
  r.all_pages = (r.len + a.page_tokens - 1) / a.page_tokens;
  r.writes = r.kept % a.page_tokens != 0 && r.len > r.kept;
  return r;
}

__device__ __forceinline__ int page_or_none(const PagesArgs& a, int page) {
  return (uint32_t)page < (uint32_t)a.num_pages ? page : -1;
}

// Entries of a row that its parent's tokens keep, and what they say of the pages.
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_keep(PagesArgs a, uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  if (j >= a.max_pages) return;
  const Row r = step_row(a, i);
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
  int found = 0;
  for (int p0 = 0; p0 < num_pages && found < want; p0 += 4 * kOneBlock) {
    const int p = p0 + 4 * (int)threadIdx.x;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = p + e < num_pages ? words[p + e] : 1u;
    int n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) n += w[e] == 0;
    int total;
    int at = found + block_prefix<kOneWaves>(n, s_wave, &total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
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
// shares and will write to, then those of tokens that begin a page.
__global__ __launch_bounds__(kOneBlock) void k_kv_pages_give(PagesArgs a, const uint32_t* words,
                                                             int32_t* list, int2* places) {
  __shared__ int s_wave[kOneWaves];
  const int tid = threadIdx.x;
  int want = 0, copies = 0;
  for (int i0 = 0; i0 < a.num_rows; i0 += kOneBlock) {
    const int i = i0 + tid;
    int copy = 0, need = 0;
    if (i < a.num_rows) {
      const Row r = step_row(a, i);
      a.out_lens[i] = r.len;
      if (r.writes) {
        const int page = a.out_table[(int64_t)i * a.max_pages + r.pages - 1];
        copy = page >= 0 && words[page] != (uint32_t)(a.num_rows - i);
      }
      need = copy + r.all_pages - r.pages;
    }
    int total;
    const int at = want + block_prefix<kOneWaves>(need, s_wave, &total);
    want += total;
    const int rank = copies + block_prefix<kOneWaves>(copy, s_wave, &total);
    copies += total;
    if (i < a.num_rows) places[i] = int2{at, copy ? rank : -1};
  }
  const int have = list_free(words, a.num_pages, want, list, s_wave);
  int done = 0;
  for (int i0 = 0; i0 < a.num_rows; i0 += kOneBlock) {
    const int i = i0 + tid;
    int made = 0;
    if (i < a.num_rows) {
      const Row r = step_row(a, i);
      const int2 place = places[i];
      int32_t* const row = a.out_table + (int64_t)i * a.max_pages;
      int at = place.x;
      if (place.y >= 0) {
        const int from = row[r.pages - 1], to = at < have ? list[at] : -1;
        row[r.pages - 1] = to;
        ++at;
        if (to >= 0) {
          int32_t* const c = a.copies + 3 * (int64_t)place.y;
          c[0] = from;
          c[1] = to;
          c[2] = r.kept % a.page_tokens;
          made = 1;
        }
      }
      for (int j = r.pages; j < r.all_pages; ++j, ++at) row[j] = at < have ? list[at] : -1;
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
  }
}

// Compaction: pages named by a row.
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_used(PagesArgs a, uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  const int len = min(max(a.seq_lens[i], 0), a.max_pages * a.page_tokens);
  if (j >= (len + a.page_tokens - 1) / a.page_tokens) return;
  const int page = page_or_none(a, a.page_table[(int64_t)i * a.max_pages + j]);
  if (page >= 0) __hip_atomic_store(words + page, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The k-th used page at or past the number of used ones goes to the k-th free one
// below it; words become the pages' new places.
__global__ __launch_bounds__(kOneBlock) void k_kv_pages_plan(PagesArgs a, uint32_t* words,
                                                             int32_t* list) {
  __shared__ int s_wave[kOneWaves];
  const int tid = threadIdx.x;
  int live = 0, total;
  for (int p0 = 0; p0 < a.num_pages; p0 += kOneBlock) {
    const int p = p0 + tid;
    block_prefix<kOneWaves>(p < a.num_pages && words[p] != 0, s_wave, &total);
    live += total;
  }
  list_free(words, live, live, list, s_wave);
  int moves = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kOneBlock) {
    const int p = p0 + tid;
    const bool used = p < a.num_pages && words[p] != 0, moved = used && p >= live;
    const int rank = moves + block_prefix<kOneWaves>(moved, s_wave, &total);
    moves += total;
    if (used) words[p] = moved ? (uint32_t)list[rank] : (uint32_t)p;
    if (moved) {
      int32_t* const c = a.copies + 3 * (int64_t)rank;
      c[0] = p;
      c[1] = list[rank];
      c[2] = a.page_tokens;
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
__global__ __launch_bounds__(kBlockThreads) void k_kv_pages_rename(PagesArgs a,
                                                                   const uint32_t* words) {
  const int i = blockIdx.y, j = blockIdx.x * kBlockThreads + threadIdx.x;
  if (j >= a.max_pages) return;
  const int len = min(max(a.seq_lens[i], 0), a.max_pages * a.page_tokens);
  const int64_t at = (int64_t)i * a.max_pages + j;
  int page = -1;
  if (j < (len + a.page_tokens - 1) / a.page_tokens) page = page_or_none(a, a.page_table[at]);
  a.out_table[at] = page < 0 ? -1 : (int)words[page];
}

// Copies of pages. An item is a head's keys or values of one page: its blocks stand
// one after the other.
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

int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

}  // namespace

// words [num_pages], list [num_pages], places [num_rows]
size_t kv_pages_workspace_bytes(const PagesArgs& a) {
  return (size_t)(2 * pad4(a.num_pages) + 2 * (int64_t)a.num_rows) * 4;
}

hipError_t launch_kv_pages_step(const PagesArgs& a, void* ws, hipStream_t s) {
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
