// Host-side driver for the argument checks of beam selection, page tables and attention
// over chosen pages, built with the host address and undefined-behaviour sanitizers
// (tests/test_generation_host_sanitizers.py). Every call fails its checks before it
// touches memory or a device, or has nothing to do; the fake device addresses are never
// dereferenced. Prints "ALL OK" and exits 0 when every status matches.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "i8mm.h"

static int failures = 0;

static void expect(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAIL %s: %s\n", what, i8mm_last_error());
    ++failures;
  }
}

template <class T>
static T* fake(uintptr_t a) { return reinterpret_cast<T*>(a); }

int main() {
  const int64_t extremes[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 15, 48, 1 << 20, 1ll << 31,
                              1ll << 40, 1ll << 62, std::numeric_limits<int64_t>::max()};
  auto* ints = fake<int32_t>(0x10000);
  auto* other = fake<int32_t>(0x7000000000);
  auto* floats = fake<float>(0x20000);
  auto* halfs = fake<uint16_t>(0x30000);

  // beam selection: pairs of sizes at their extremes, without a workspace or outputs
  for (int f = 0; f < 5; ++f)
    for (int g = 0; g < 5; ++g)
      for (int64_t u : extremes)
        for (int64_t w : extremes) {
          int64_t size[] = {2, 3, 100, 3, 100};   // batch, beams, vocab, count, row_stride
          size[f] = u;
          size[g] = w;
          const size_t need = i8mm_beam_select_workspace_bytes(0, size[0], size[1], size[2], size[3]);
          (void)i8mm_beam_select_workspace_bytes(1, size[0], size[1], size[2], size[3]);
          if (size[0] == 0) continue;   // nothing to do
          expect(i8mm_beam_select(floats, 1, size[4], floats, nullptr, size[0], size[1], size[2], size[3],
                                  -1, nullptr, ints, ints, ints, nullptr, 0, nullptr) < 0, "beam outputs");
          if (need > 0)
            expect(i8mm_beam_select(floats, 0, size[4], floats, nullptr, size[0], size[1], size[2],
                                    size[3], -1, floats, ints, ints, ints, nullptr, 0, nullptr) < 0,
                   "beam workspace");
        }
  for (int32_t eos : {std::numeric_limits<int32_t>::min(), -2, 100, std::numeric_limits<int32_t>::max()})
    expect(i8mm_beam_select(floats, 0, 100, floats, nullptr, 2, 3, 100, 3, eos, floats, ints, ints, ints,
                            floats, 1 << 20, nullptr) == I8MM_EINVAL, "beam eos");

  // page tables
  for (int f = 0; f < 6; ++f)
    for (int g = 0; g < 6; ++g)
      for (int64_t u : extremes)
        for (int64_t w : extremes) {
          int64_t size[] = {3, 5, 4, 20, 64, 1};   // seqs, width, rows, pages, page_tokens, new
          size[f] = u;
          size[g] = w;
          (void)i8mm_kv_pages_workspace_bytes(size[2], size[1], size[3]);
          expect(i8mm_kv_pages_step(ints, ints, size[0], size[1], ints, ints, nullptr, size[5], size[2],
                                    size[3], size[4], other, other, other, nullptr, floats, 1ull << 62,
                                    nullptr) < 0, "step counts");
          expect(i8mm_kv_pages_compact(ints, ints, size[0], size[1], size[3], size[4], ints, ints, nullptr,
                                       floats, 1ull << 62, nullptr) < 0, "compact counts");
          if (i8mm_kv_pages_workspace_bytes(size[2], size[1], size[3]) > 0)
            expect(i8mm_kv_pages_step(ints, ints, size[0], size[1], ints, ints, nullptr, size[5], size[2],
                                      size[3], size[4], other, other, other, other, nullptr, 0,
                                      nullptr) < 0, "step workspace");
          const i8mm_kv_cache c = {fake<int8_t>(0x10000), floats, fake<int8_t>(0x10000), floats,
                                   size[3], size[4], size[0], size[1]};
          if (size[2] != 0)   // (no copies: nothing to do)
            expect(int8_kv_cache_copy_pages(&c, nullptr, nullptr, ints, size[2], nullptr) < 0, "copies");
        }
  expect(int8_kv_cache_copy_pages(nullptr, nullptr, ints, ints, 1, nullptr) == I8MM_EINVAL, "copy null");

  // chosen pages
  for (int f = 0; f < 12; ++f)
    for (int g = 0; g < 12; ++g)
      for (int64_t u : extremes)
        for (int64_t w : extremes) {
          i8mm_kv_cache c = {fake<int8_t>(0x10000), floats, fake<int8_t>(0x10000), floats, 8, 64, 2, 64};
          i8mm_kv_batch b = {ints, ints, ints, 2, 4, 6, 4, 256};
          int64_t count = 3, first = 1, recent = 1;
          int64_t* size[] = {&c.num_pages, &c.page_tokens, &c.kv_heads, &c.head_dim, &b.num_seqs,
                             &b.max_pages, &b.total_tokens, &b.max_tokens, &b.max_len, &count, &first,
                             &recent};
          *size[f] = u;
          *size[g] = w;
          for (int64_t heads : {(int64_t)4, (int64_t)65534, (int64_t)1 << 40})
            (void)int8_kv_cache_attention_pages_workspace_bytes(&c, &b, heads, count);
          if (b.total_tokens == 0) continue;   // nothing to do
          expect(int8_kv_cache_select_pages(halfs, 256, 64, 4, &c, halfs, &b, nullptr, count, first, recent,
                                            nullptr, nullptr) < 0, "select output");
          expect(int8_kv_cache_attention_pages(halfs, 256, 64, 4, &c, &b, nullptr, nullptr, count, 1.f,
                                               halfs, nullptr, 0, nullptr) < 0, "attention lists");
          if (c.num_pages > 0)
            expect(int8_kv_cache_page_means(&c, &b, nullptr, nullptr) < 0, "means");
        }
  if (failures == 0) std::printf("ALL OK\n");
  return failures != 0;
}
