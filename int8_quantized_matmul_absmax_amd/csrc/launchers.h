// Internal launch wrappers of the i8mm kernels. Arguments are validated by
// the C-ABI layer before these are called; each returns the hipError_t of its
// launch(es).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "i8mm.h"

namespace i8mm {

hipError_t launch_fill_u32(uint32_t* p, int64_t count, uint32_t value, hipStream_t s);

// tau16: smallest fp16 magnitude bit pattern (sign cleared) whose value is
// >= the threshold (0 for a threshold <= 0, 0x7c00 above the largest finite
// fp16); see fp16_threshold_pattern.
hipError_t launch_outlier_flags(const uint16_t* X, int64_t M, int64_t K, uint32_t tau16,
                                uint32_t* bitmap, hipStream_t s);

uint32_t fp16_threshold_pattern(float threshold);

hipError_t launch_cols_from_bitmap(const uint32_t* bitmap, int64_t K, int32_t* cols,
                                   int32_t* n_out, hipStream_t s);

// The layer's detection without a cleared bitmap: part[b][w] (bands x
// ceil(K/32) words, every word written) holds the flags of row band b, rows
// [b * ceil(M/bands), ...); the bitmap is their OR. flag_bands(M, K) is the
// band count the layer uses (1 .. kMaxFlagBands, no band empty).
constexpr int kMaxFlagBands = 16;
int flag_bands(int64_t M, int64_t K);
hipError_t launch_outlier_flag_bands(const uint16_t* X, int64_t M, int64_t K, uint32_t tau16,
                                     int bands, uint32_t* part, hipStream_t s);

// Row pass over X (or W): optional absmax quantization (Xq, sx), optional
// gather of outlier columns (Xo), optional cols/n output from the first row's
// block. bitmap == nullptr means no outlier columns.
hipError_t launch_rows(const uint16_t* X, int64_t M, int64_t K, const uint32_t* bitmap,
                       int8_t* Xq, float* sx, uint16_t* Xo, int32_t* cols, int32_t* n_out,
                       hipStream_t s);
// The same with the flags given as `bands` partial bitmaps (bands x
// ceil(K/32) words, see launch_outlier_flag_bands); the first block also
// writes their OR to bitmap_out when it is given, and, when kbl is given,
// the list of 64-column k-blocks that hold a normal column (kbl[0] = count,
// then the blocks ascending; 1 + ceil(K/64) ints).
hipError_t launch_rows_banded(const uint16_t* X, int64_t M, int64_t K, const uint32_t* flags,
                              int bands, uint32_t* bitmap_out, int8_t* Xq, float* sx,
                              uint16_t* Xo, int32_t* cols, int32_t* n_out, int32_t* kbl,
                              hipStream_t s);

// Wo: the fp16 outlier weight columns [N, LD(n)] written by
// launch_recover_outlier_w (or launch_gather_w_cols) with room for wo_cols
// columns, or nullptr; with 16 < n <= wo_cols and Wo given, the outlier
// product runs as a second main-loop segment over them. Xd, bmp: the
// layer's X [M, K] and its outlier bitmap, or nullptr; given, more than 16
// outlier columns that Wo does not take run as the dense second segment over
// all K columns. Otherwise the outlier product runs in the epilogue. Wf: the
// fp16 weight [N, K] when the layer keeps one (its columns are the outlier
// weights), or nullptr (they are recovered from Wq and sw).
// kbl: the k-block list of launch_rows_banded, or nullptr; given, the
// int8 loop of the segment modes visits only those k-blocks.
hipError_t launch_gemm(const int8_t* Xq, const int8_t* Wq, const float* sx, const float* sw,
                       int64_t M, int64_t N, int64_t K, const uint16_t* Xo,
                       const int32_t* cols, const int32_t* n_out, const uint16_t* bias,
                       uint16_t* Y, int32_t* C, const uint16_t* Wo, int wo_cols,
                       const uint16_t* Wf, const uint16_t* Xd, const uint32_t* bmp,
                       const int32_t* kbl, hipStream_t s);

// Wo[j, t] = fp16(fl32(fl32(Wq[j, cols[t]] * sw[j]) / 127)) for t < n, +0.0 up
// to LD(n); nothing when n <= 16 or n > wo_cols (n read on the device).
hipError_t launch_recover_outlier_w(const int8_t* Wq, const float* sw, int64_t N, int64_t K,
                                    const int32_t* cols, const int32_t* n_out, int wo_cols,
                                    uint16_t* Wo, hipStream_t s);

// Wo[j, t] = Wf[j, cols[t]] (the fp16 weight's own columns) for t < n, +0.0
// up to LD(n); nothing when n <= 16 or n > wo_cols (n read on the device).
hipError_t launch_gather_w_cols(const uint16_t* Wf, int64_t N, int64_t K, const int32_t* cols,
                                const int32_t* n_out, int wo_cols, uint16_t* Wo, hipStream_t s);

// The whole layer in one launch for 1 <= M <= 16 tokens whose codes fit in
// LDS (decode_applies): detection, row quantization and the few-token
// matmul with its epilogue. Writes the same intermediates as the separate
// kernels (bitmap, cols, n, sx, Xq, Xo with leading dimension LD(n)) and Y.
// Wf: the fp16 weight when the layer keeps one, else nullptr.
bool decode_applies(int64_t M, int64_t K);
hipError_t launch_decode(const uint16_t* X, const int8_t* Wq, const float* sw, int64_t M,
                         int64_t N, int64_t K, uint32_t tau16, const uint16_t* bias, uint16_t* Y,
                         const uint16_t* Wf, uint32_t* bitmap, int32_t* cols, int32_t* n_out,
                         float* sx, int8_t* Xq, uint16_t* Xo, hipStream_t s);

// Few-token form of launch_gemm (same arguments and results), used for
// 1 <= M <= 64.
bool gemv_applies(int64_t M);
hipError_t launch_gemv(const int8_t* Xq, const int8_t* Wq, const float* sx, const float* sw,
                       int64_t M, int64_t N, int64_t K, const uint16_t* Xo,
                       const int32_t* cols, const int32_t* n_out, const uint16_t* bias,
                       uint16_t* Y, int32_t* C, const uint16_t* Wf, hipStream_t s);

// ---- paged 8-bit key/value cache
// The cache and batch structs of the C ABI narrowed to what kernels index
// with, arguments validated: slots = page_tokens / 16 blocks a page, len_cap =
// min(max_len, max_pages * page_tokens).
struct KvArgs {
  int8_t* k_codes;
  float* k_absmax;
  int8_t* v_codes;
  float* v_absmax;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;   // or nullptr: one token a sequence
  int num_pages, slots, kv_heads, head_dim;
  int num_seqs, max_pages, total_tokens, max_tokens, len_cap;
};
struct RotaryArgs {
  const float* cos;           // nullptr: no rotation
  const float* sin;
  int dim, interleaved;
};

bool kv_head_dim_ok(int64_t D);

hipError_t launch_kv_append(const uint16_t* k, int64_t k_ts, int64_t k_hs, const uint16_t* v,
                            int64_t v_ts, int64_t v_hs, const KvArgs& a, const RotaryArgs& r,
                            hipStream_t s);
hipError_t launch_kv_read(const KvArgs& a, uint16_t* k, uint16_t* v, hipStream_t s);

struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const float* slopes;        // or nullptr
  uint16_t* out;
  float* part;                // workspace of attn_workspace_bytes
  float scale_log2;           // scale * log2(e)
  int q_heads, causal, window;
};
size_t attn_workspace_bytes(const KvArgs& a, int q_heads);
hipError_t launch_kv_attention(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t,
                               hipStream_t s);

// ---- a beam search's choice of its next beams (arguments as in the C ABI)
struct BeamArgs {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  const int32_t* live;        // or nullptr: all
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  int32_t* out_live;
  void* ws;
  int64_t vocab;
  int fp32, batch, beams, count, eos;
};
size_t beam_workspace_bytes(const BeamArgs& a);
hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s);

// Threads of a launch along x stay below 2^32.
constexpr int64_t max_grid(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

// Attention over the `count` pages that each token and key/value head lists.
size_t attn_pages_workspace_bytes(const KvArgs& a, int q_heads, int count);
bool attn_pages_fits(const KvArgs& a, int q_heads, int count);   // one launch
hipError_t launch_kv_attention_pages(const KvArgs& a, const RotaryArgs& r, const AttnArgs& t,
                                     const int32_t* chosen, int count, hipStream_t s);
// Mean keys of the pages that hold the batch's new tokens, and the choice of pages.
constexpr int kMaxSelectPages = I8MM_MAX_SELECT_PAGES;
// Threads of a block of the choice, given its blocks and the candidates of one: 1024
// where a compute unit has one block, which is with few blocks, and where keys fill its LDS
// (means and choice, with 256 and 1024 threads). 8 blocks of 509 candidates 15.4 and
// 16.1 us, of 1021 21.0 and 17.6, of 2045 31.2 and 23.0; 256 of 1021 27.7 and 24.4, 320 32.4
// and 35.1, 512 35.2 and 39.6; 2048 of 4093 105 and 107, of 8189 170 and 121; 16384 of
// 1997 516 and 778. And 256 for blocks that would be too many for a launch with 1024.
constexpr int select_threads(int64_t blocks, int64_t candidates) {
  return candidates > 512 && (blocks <= 256 || candidates > 4096) && blocks <= max_grid(1024) ? 1024 : 256;
}
int64_t page_means_tasks(const KvArgs& a);   // waves for a sequence, four a block
hipError_t launch_kv_page_means(const KvArgs& a, uint16_t* means, hipStream_t s);
hipError_t launch_kv_select_pages(const KvArgs& a, const RotaryArgs& r, const uint16_t* q, int64_t q_ts,
                                  int64_t q_hs, int q_heads, const uint16_t* means, int count, int first,
                                  int recent, int32_t* out, hipStream_t s);

// ---- pages of the key/value cache (arguments as in the C ABI)
struct PagesArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* parents;
  const int32_t* keep;        // or nullptr: all tokens
  const int32_t* new_tokens;  // or nullptr: new_all
  int32_t* out_table;
  int32_t* out_lens;
  int32_t* copies;
  int32_t* counts;
  int32_t* batch_lens;        // or nullptr, then full too
  int32_t* full;
  int num_seqs, max_pages, num_rows, num_pages, page_tokens, new_all, max_len;
};
size_t kv_pages_workspace_bytes(const PagesArgs& a, int rows);   // of the step or the compaction
hipError_t launch_kv_pages_step(const PagesArgs& a, void* ws, hipStream_t s);
hipError_t launch_kv_pages_compact(const PagesArgs& a, void* ws, hipStream_t s);
// (of KvArgs the cache's part)
hipError_t launch_kv_copy_pages(const KvArgs& a, uint16_t* means, const int32_t* copies,
                                const int32_t* count, int most, hipStream_t s);

hipError_t launch_gelu(const uint16_t* X, int64_t count, uint16_t* Y, hipStream_t s);

}  // namespace i8mm
