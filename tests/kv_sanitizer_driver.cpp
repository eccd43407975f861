// Host-side driver for the key/value cache calls' argument checks, built with the
// host address and undefined-behaviour sanitizers
// (tests/test_kv_host_sanitizers.py). Every call fails its checks before it
// touches memory or a device, or has nothing to do; the fake device addresses are
// never dereferenced. Prints "ALL OK" and exits 0 when every status matches.
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

static i8mm_kv_cache cache() {
  return {fake<int8_t>(0x10000), fake<float>(0x20000), fake<int8_t>(0x30000), fake<float>(0x40000),
          8, 64, 2, 64};
}
static i8mm_kv_batch batch() {
  return {fake<int32_t>(0x50000), fake<int32_t>(0x60000), fake<int32_t>(0x70000), 2, 4, 6, 4, 256};
}

static int attention(const i8mm_kv_cache* c, const i8mm_kv_batch* b, int64_t heads = 4,
                     float scale = 1.f, int64_t stride = 64, const i8mm_rotary* r = nullptr) {
  auto* x = fake<uint16_t>(0x80000);
  return int8_kv_cache_attention(x, 4 * stride, stride, heads, c, b, r, scale, 1, 0, nullptr, x,
                                 nullptr, 0, nullptr);
}

int main() {
  const int64_t extremes[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 15, 1 << 20, 1ll << 31,
                              1ll << 40, 1ll << 62, std::numeric_limits<int64_t>::max()};
  auto* x = fake<uint16_t>(0x80000);
  // one size of the structs at a time at every extreme, and pairs of them, for
  // calls that cannot reach the device: without a workspace, or without tokens
  for (int f = 0; f < 9; ++f)
    for (int g = 0; g < 9; ++g)
      for (int64_t u : extremes)
        for (int64_t w : extremes) {
          i8mm_kv_cache c = cache();
          i8mm_kv_batch b = batch();
          int64_t* size[] = {&c.num_pages, &c.page_tokens, &c.kv_heads, &c.head_dim, &b.num_seqs,
                             &b.max_pages, &b.total_tokens, &b.max_tokens, &b.max_len};
          *size[f] = u;
          *size[g] = w;
          for (int64_t heads : {(int64_t)4, (int64_t)65534, (int64_t)1 << 40})
            (void)int8_kv_cache_attention_workspace_bytes(&c, &b, heads);
          c.k_codes = nullptr;   // refused if there are pages, whatever else holds
          if (c.num_pages <= 0) continue;
          expect(int8_kv_cache_append(x, 128, 64, x, 128, 64, &c, &b, nullptr, nullptr) < 0, "append");
          expect(attention(&c, &b) < 0, "attention");
          expect(int8_kv_cache_read(&c, &b, x, x, nullptr) < 0, "read");
        }
  i8mm_kv_cache c = cache();
  i8mm_kv_batch b = batch();
  expect(int8_kv_cache_append(x, 128, 64, x, 128, 64, nullptr, &b, nullptr, nullptr) == I8MM_EINVAL,
         "append null cache");
  expect(attention(&c, nullptr) == I8MM_EINVAL, "attention null batch");
  expect(int8_kv_cache_read(nullptr, nullptr, x, x, nullptr) == I8MM_EINVAL, "read nulls");
  expect(int8_kv_cache_attention_workspace_bytes(nullptr, nullptr, 4) == 0, "workspace nulls");
  for (int64_t h : extremes)
    if (h != 1 << 20 && (h <= 0 || h > 65535 || h % 2 != 0))
      expect(attention(&c, &b, h) == I8MM_EINVAL, "attention heads");
  for (float s : {0.f, -1.f, std::nanf(""), INFINITY})
    expect(attention(&c, &b, 4, s) == I8MM_EINVAL, "attention scale");
  expect(attention(&c, &b, 4, 1.f, 65) == I8MM_EALIGN, "attention stride");
  expect(attention(&c, &b, 4, 1.f, -64) == I8MM_EINVAL, "attention negative stride");
  for (int64_t u : extremes) {
    const i8mm_rotary dims = {fake<float>(0x90000), fake<float>(0x90000), u, 256, 0};
    expect(attention(&c, &b, 4, 1.f, 64, &dims) == I8MM_EINVAL, "rotary dim");
    const i8mm_rotary rows = {nullptr, fake<float>(0x90000), 64, u, 0};
    expect(attention(&c, &b, 4, 1.f, 64, &rows) < 0, "rotary positions");
  }
  // rows and workspaces that 64 bits would not hold
  b.total_tokens = std::numeric_limits<int32_t>::max();
  b.max_len = 1 << 30;
  b.max_pages = 1 << 24;
  expect(int8_kv_cache_attention_workspace_bytes(&c, &b, 65534) == 0, "workspace overflow");
  expect(attention(&c, &b, 65534) == I8MM_EINVAL, "attention overflow");
  b.max_tokens = 1 << 28;
  expect(attention(&c, &b, 20) == I8MM_EINVAL, "attention rows");
  // no tokens: nothing to do, and no device needed
  b = batch();
  b.total_tokens = b.num_seqs = 0;
  expect(int8_kv_cache_append(nullptr, 128, 64, nullptr, 128, 64, &c, &b, nullptr, nullptr) == I8MM_OK,
         "append nothing");
  expect(int8_kv_cache_read(&c, &b, nullptr, nullptr, nullptr) == I8MM_OK, "read nothing");
  if (failures == 0) std::printf("ALL OK\n");
  return failures != 0;
}
