// C-ABI of the i8mm library: argument validation, workspace layout and the
// launch sequence of each entry point. Declarations and the contract of each
// call are in include/i8mm.h.

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "i8mm.h"
#include "launchers.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return I8MM_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_state[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

int check_device() {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(I8MM_ENODEVICE, "no HIP device: %s", hipGetErrorString(e));
  if (dev >= 0 && dev < kMaxDevices) {
    int st = g_dev_state[dev].load(std::memory_order_acquire);
    if (st == 1) return I8MM_OK;
    if (st == 2) return fail(I8MM_ENODEVICE, "device %d is not gfx950", dev);
  }
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess)
    return fail(I8MM_ENODEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
  const bool good = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev >= 0 && dev < kMaxDevices) g_dev_state[dev].store(good ? 1 : 2, std::memory_order_release);
  if (!good) return fail(I8MM_ENODEVICE, "device %d is %s, not gfx950", dev, prop.gcnArchName);
  return I8MM_OK;
}

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(I8MM_ELAUNCH, "%s: %s", what, hipGetErrorString(e));
  return I8MM_OK;
}

#define I8MM_TRY(expr)        \
  do {                        \
    int _st = (expr);         \
    if (_st != I8MM_OK) return _st; \
  } while (0)

// Common shape checks: sizes non-negative and within int32 row/column counts,
// K a multiple of 16 and within the int32 accumulation bound.
int check_dims(const char* fn, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return fail(I8MM_EINVAL, "%s: negative size", fn);
  if (M > INT32_MAX || N > INT32_MAX) return fail(I8MM_EINVAL, "%s: size beyond int32", fn);
  if (K % 16 != 0) return fail(I8MM_EALIGN, "%s: K=%lld is not a multiple of 16", fn, (long long)K);
  if (K > I8MM_MAX_K) return fail(I8MM_ERANGE, "%s: K=%lld exceeds %d", fn, (long long)K, I8MM_MAX_K);
  return I8MM_OK;
}

int check_ptr(const char* fn, const char* name, const void* p, bool required) {
  if (!p) return required ? fail(I8MM_EINVAL, "%s: %s is NULL", fn, name) : I8MM_OK;
  if (!aligned16(p)) return fail(I8MM_EALIGN, "%s: %s is not 16-byte aligned", fn, name);
  return I8MM_OK;
}

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Workspace of linear_int8_mixed: bitmap | cols | n | sx | Xq | Xo |
// partial flag words (kMaxFlagBands x ceil(K/32), at *part when given) |
// the GEMM's k-block list (1 + ceil(K/64) ints, at *kbl when given).
bool layout(int64_t M, int64_t K, int64_t* off, int64_t* part = nullptr,
            int64_t* kbl = nullptr) {
  if (M < 0 || K < 0 || K % 16 != 0 || K > I8MM_MAX_K || M > INT32_MAX) return false;
  int64_t p = 0;
  off[0] = p; p = round_up(p + (K + 31) / 32 * 4, kAlign);
  off[1] = p; p = round_up(p + K * 4, kAlign);
  off[2] = p; p = round_up(p + 4, kAlign);
  off[3] = p; p = round_up(p + M * 4, kAlign);
  off[4] = p; p = round_up(p + M * K, kAlign);
  off[5] = p; p = round_up(p + M * I8MM_OUTLIER_LD(K) * 2, kAlign);
  if (part) *part = p;
  p = round_up(p + i8mm::kMaxFlagBands * ((K + 31) / 32) * 4, kAlign);
  if (kbl) *kbl = p;
  p = round_up(p + (1 + (K + 63) / 64) * 4, kAlign);
  off[6] = p;
  return true;
}

// Bytes of the region of linear_int8_mixed_workspace_bytes_many_outliers
// after the minimal workspace: the recovered fp16 outlier weight columns
// for up to I8MM_OUTLIER_REGION_COLS outlier columns.
int64_t wo_region_bytes(int64_t N, int64_t K) {
  return round_up(N * I8MM_OUTLIER_LD(std::min<int64_t>(K, I8MM_OUTLIER_REGION_COLS)) * 2, kAlign);
}

}  // namespace

extern "C" {

const char* i8mm_last_error(void) { return g_err; }

const char* i8mm_status_string(int status) {
  switch (status) {
    case I8MM_OK: return "I8MM_OK";
    case I8MM_EINVAL: return "I8MM_EINVAL";
    case I8MM_EALIGN: return "I8MM_EALIGN";
    case I8MM_EWORKSPACE: return "I8MM_EWORKSPACE";
    case I8MM_ENODEVICE: return "I8MM_ENODEVICE";
    case I8MM_ELAUNCH: return "I8MM_ELAUNCH";
    case I8MM_ERANGE: return "I8MM_ERANGE";
    default: return "I8MM_UNKNOWN";
  }
}

size_t linear_int8_mixed_workspace_bytes(int64_t M, int64_t K) {
  int64_t off[7];
  return layout(M, K, off) ? (size_t)off[6] : 0;
}

size_t linear_int8_mixed_workspace_bytes_many_outliers(int64_t M, int64_t K, int64_t N) {
  int64_t off[7];
  if (N < 0 || N > INT32_MAX || !layout(M, K, off)) return 0;
  return (size_t)(off[6] + wo_region_bytes(N, K));
}

int i8mm_workspace_layout(int64_t M, int64_t K, int64_t* offsets) {
  if (!offsets) return fail(I8MM_EINVAL, "i8mm_workspace_layout: offsets is NULL");
  if (!layout(M, K, offsets)) return fail(I8MM_EINVAL, "i8mm_workspace_layout: invalid sizes");
  return ok();
}

int int8_quantize_colwise_weight(const uint16_t* W, int64_t N, int64_t K, int8_t* Wq, float* sw,
                                 i8mm_stream_t stream) {
  const char* fn = "int8_quantize_colwise_weight";
  I8MM_TRY(check_dims(fn, N, 0, K));
  I8MM_TRY(check_ptr(fn, "W", W, N * K > 0));
  I8MM_TRY(check_ptr(fn, "Wq", Wq, N * K > 0));
  I8MM_TRY(check_ptr(fn, "sw", sw, N > 0));
  if (N == 0) return ok();
  I8MM_TRY(check_device());
  hipStream_t s = (hipStream_t)stream;
  I8MM_TRY(launched(i8mm::launch_rows(W, N, K, nullptr, Wq, sw, nullptr, nullptr, nullptr, s), fn));
  return ok();
}

int int8_quantize_rowwise(const uint16_t* X, int64_t M, int64_t K, const uint32_t* outlier_bitmap,
                          int8_t* Xq, float* sx, i8mm_stream_t stream) {
  const char* fn = "int8_quantize_rowwise";
  I8MM_TRY(check_dims(fn, M, 0, K));
  I8MM_TRY(check_ptr(fn, "X", X, M * K > 0));
  I8MM_TRY(check_ptr(fn, "outlier_bitmap", outlier_bitmap, false));
  I8MM_TRY(check_ptr(fn, "Xq", Xq, M * K > 0));
  I8MM_TRY(check_ptr(fn, "sx", sx, M > 0));
  if (M == 0) return ok();
  I8MM_TRY(check_device());
  hipStream_t s = (hipStream_t)stream;
  I8MM_TRY(launched(
      i8mm::launch_rows(X, M, K, outlier_bitmap, Xq, sx, nullptr, nullptr, nullptr, s), fn));
  return ok();
}

int outlier_detect_gather(const uint16_t* X, int64_t M, int64_t K, float threshold,
                          uint32_t* bitmap, int32_t* cols, int32_t* n_outliers, uint16_t* Xo,
                          i8mm_stream_t stream) {
  const char* fn = "outlier_detect_gather";
  I8MM_TRY(check_dims(fn, M, 0, K));
  if (std::isnan(threshold)) return fail(I8MM_EINVAL, "%s: threshold is NaN", fn);
  I8MM_TRY(check_ptr(fn, "X", X, M * K > 0));
  I8MM_TRY(check_ptr(fn, "bitmap", bitmap, K > 0));
  I8MM_TRY(check_ptr(fn, "cols", cols, K > 0));
  I8MM_TRY(check_ptr(fn, "n_outliers", n_outliers, true));
  I8MM_TRY(check_ptr(fn, "Xo", Xo, false));
  I8MM_TRY(check_device());
  hipStream_t s = (hipStream_t)stream;
  const int64_t nwords = (K + 31) / 32;
  I8MM_TRY(launched(i8mm::launch_fill_u32(bitmap, nwords, 0u, s), fn));
  if (M > 0) I8MM_TRY(launched(i8mm::launch_outlier_flags(X, M, K, i8mm::fp16_threshold_pattern(threshold), bitmap, s), fn));
  I8MM_TRY(launched(i8mm::launch_cols_from_bitmap(bitmap, K, cols, n_outliers, s), fn));
  if (Xo && M > 0)
    I8MM_TRY(launched(
        i8mm::launch_rows(X, M, K, bitmap, nullptr, nullptr, Xo, nullptr, nullptr, s), fn));
  return ok();
}

int int8_mm_dequant(const int8_t* Xq, const int8_t* Wq, const float* sx, const float* sw,
                    int64_t M, int64_t N, int64_t K, const uint16_t* Xo, const int32_t* cols,
                    const int32_t* n_outliers, const uint16_t* bias, uint16_t* Y, int32_t* C,
                    i8mm_stream_t stream) {
  const char* fn = "int8_mm_dequant";
  I8MM_TRY(check_dims(fn, M, N, K));
  I8MM_TRY(check_ptr(fn, "Xq", Xq, M * K > 0));
  I8MM_TRY(check_ptr(fn, "Wq", Wq, N * K > 0));
  I8MM_TRY(check_ptr(fn, "sx", sx, M > 0));
  I8MM_TRY(check_ptr(fn, "sw", sw, N > 0));
  const bool any_o = Xo || cols || n_outliers;
  const bool all_o = Xo && cols && n_outliers;
  if (any_o && !all_o)
    return fail(I8MM_EINVAL, "%s: Xo, cols and n_outliers must be given together", fn);
  I8MM_TRY(check_ptr(fn, "Xo", Xo, false));
  I8MM_TRY(check_ptr(fn, "cols", cols, false));
  I8MM_TRY(check_ptr(fn, "n_outliers", n_outliers, false));
  I8MM_TRY(check_ptr(fn, "bias", bias, false));
  I8MM_TRY(check_ptr(fn, "Y", Y, false));
  I8MM_TRY(check_ptr(fn, "C", C, false));
  if (!Y && !C) return fail(I8MM_EINVAL, "%s: neither Y nor C given", fn);
  if (M == 0 || N == 0) return ok();
  I8MM_TRY(check_device());
  hipStream_t s = (hipStream_t)stream;
  I8MM_TRY(launched(
      i8mm::launch_gemm(Xq, Wq, sx, sw, M, N, K, Xo, cols, n_outliers, bias, Y, C, nullptr, 0,
                        nullptr, nullptr, nullptr, nullptr, s),
      fn));
  return ok();
}

}  // extern "C"

namespace {

// The activation side of the layer (steps a1-a3) into the workspace:
// detection as per-band partial flags (no clearing launch), then the row
// pass, which ORs them, writes the bitmap, cols, n and the GEMM's k-block
// list, gathers the outlier columns into Xo and quantizes the normal part
// into Xq, sx.
int x_side(const char* fn, const uint16_t* X, int64_t M, int64_t K, uint32_t tau16, char* ws,
           const int64_t* off, int64_t off_part, int64_t off_kbl, hipStream_t s) {
  uint32_t* bitmap = reinterpret_cast<uint32_t*>(ws + off[0]);
  int32_t* cols = reinterpret_cast<int32_t*>(ws + off[1]);
  int32_t* n_o = reinterpret_cast<int32_t*>(ws + off[2]);
  float* sx = reinterpret_cast<float*>(ws + off[3]);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + off[4]);
  uint16_t* Xo = reinterpret_cast<uint16_t*>(ws + off[5]);
  uint32_t* part = reinterpret_cast<uint32_t*>(ws + off_part);
  int32_t* kbl = reinterpret_cast<int32_t*>(ws + off_kbl);
  const int bands = i8mm::flag_bands(M, K);
  I8MM_TRY(launched(i8mm::launch_outlier_flag_bands(X, M, K, tau16, bands, part, s), fn));
  I8MM_TRY(launched(
      i8mm::launch_rows_banded(X, M, K, part, bands, bitmap, Xq, sx, Xo, cols, n_o, kbl, s),
      fn));
  return I8MM_OK;
}

// Workspace pointer and size checks shared by the calls that take one.
int check_workspace(const char* fn, const void* workspace, size_t workspace_bytes,
                    const int64_t* off) {
  if (!workspace) return fail(I8MM_EWORKSPACE, "%s: workspace is NULL", fn);
  if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return fail(I8MM_EALIGN, "%s: workspace is not 256-byte aligned", fn);
  if ((int64_t)workspace_bytes < off[6])
    return fail(I8MM_EWORKSPACE, "%s: workspace has %zu bytes, needs %lld", fn, workspace_bytes,
                (long long)off[6]);
  return I8MM_OK;
}

// Argument checks of the layer calls (all before any device work).
int check_layer_args(const char* fn, const uint16_t* X, int64_t M, int64_t K, const int8_t* Wq,
                     const float* sw, int64_t N, const uint16_t* bias, float threshold,
                     const uint16_t* Y) {
  I8MM_TRY(check_dims(fn, M, N, K));
  if (std::isnan(threshold)) return fail(I8MM_EINVAL, "%s: threshold is NaN", fn);
  I8MM_TRY(check_ptr(fn, "X", X, M * K > 0));
  I8MM_TRY(check_ptr(fn, "Wq", Wq, N * K > 0));
  I8MM_TRY(check_ptr(fn, "sw", sw, N > 0));
  I8MM_TRY(check_ptr(fn, "bias", bias, false));
  I8MM_TRY(check_ptr(fn, "Y", Y, M * N > 0));
  return I8MM_OK;
}

// The whole layer after argument checks common to both weight modes. Wf: the
// fp16 weight when the layer keeps one (its outlier columns feed the outlier
// product), else nullptr (they are recovered from Wq, sw). quantize_w: write
// Wf's codes into Wq, sw first.
int run_layer(const char* fn, const uint16_t* X, int64_t M, int64_t K, const int8_t* Wq,
              const float* sw, int64_t N, const uint16_t* bias, float threshold, uint16_t* Y,
              void* workspace, size_t workspace_bytes, hipStream_t s, const uint16_t* Wf,
              bool quantize_w) {
  I8MM_TRY(check_layer_args(fn, X, M, K, Wq, sw, N, bias, threshold, Y));
  int64_t off[7], off_part = 0, off_kbl = 0;
  layout(M, K, off, &off_part, &off_kbl);
  I8MM_TRY(check_workspace(fn, workspace, workspace_bytes, off));
  if (M == 0 || N == 0) return ok();
  I8MM_TRY(check_device());
  char* ws = static_cast<char*>(workspace);
  uint32_t* bitmap = reinterpret_cast<uint32_t*>(ws + off[0]);
  int32_t* cols = reinterpret_cast<int32_t*>(ws + off[1]);
  int32_t* n_o = reinterpret_cast<int32_t*>(ws + off[2]);
  float* sx = reinterpret_cast<float*>(ws + off[3]);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + off[4]);
  uint16_t* Xo = reinterpret_cast<uint16_t*>(ws + off[5]);
  const uint32_t tau16 = i8mm::fp16_threshold_pattern(threshold);
  if (quantize_w)
    I8MM_TRY(launched(i8mm::launch_rows(Wf, N, K, nullptr, const_cast<int8_t*>(Wq),
                                        const_cast<float*>(sw), nullptr, nullptr, nullptr, s),
                      fn));
  if (i8mm::decode_applies(M, K)) {
    // few tokens: the whole layer in one launch
    I8MM_TRY(launched(i8mm::launch_decode(X, Wq, sw, M, N, K, tau16, bias, Y, Wf, bitmap, cols,
                                          n_o, sx, Xq, Xo, s),
                      fn));
    return ok();
  }
  I8MM_TRY(x_side(fn, X, M, K, tau16, ws, off, off_part, off_kbl, s));
  // The workspace beyond the minimal layout holds the recovered fp16 outlier
  // weight columns for the tiled GEMM, N rows of LD(n) halfs, for n up to the
  // columns it has room for (the kernels do nothing for 16 or fewer columns,
  // or for more than that room; the GEMM's dense loop takes those).
  uint16_t* Wo = nullptr;
  int wo_cols = 0;
  if (!i8mm::gemv_applies(M)) {
    const int64_t room = ((int64_t)workspace_bytes - off[6]) / (2 * N) / 32 * 32;
    if (room >= 32) {
      wo_cols = (int)std::min<int64_t>(room, I8MM_OUTLIER_LD(K));
      Wo = reinterpret_cast<uint16_t*>(ws + off[6]);
      if (Wf)
        I8MM_TRY(launched(i8mm::launch_gather_w_cols(Wf, N, K, cols, n_o, wo_cols, Wo, s), fn));
      else
        I8MM_TRY(launched(
            i8mm::launch_recover_outlier_w(Wq, sw, N, K, cols, n_o, wo_cols, Wo, s), fn));
    }
  }
  I8MM_TRY(launched(i8mm::launch_gemm(Xq, Wq, sx, sw, M, N, K, Xo, cols, n_o, bias, Y, nullptr,
                                      Wo, wo_cols, Wf, X, bitmap,
                                      reinterpret_cast<const int32_t*>(ws + off_kbl), s),
                    fn));
  return ok();
}

}  // namespace

extern "C" {

int linear_int8_mixed(const uint16_t* X, int64_t M, int64_t K, const int8_t* Wq, const float* sw,
                      int64_t N, const uint16_t* bias, float threshold, uint16_t* Y,
                      void* workspace, size_t workspace_bytes, i8mm_stream_t stream) {
  return run_layer("linear_int8_mixed", X, M, K, Wq, sw, N, bias, threshold, Y, workspace,
                   workspace_bytes, (hipStream_t)stream, nullptr, false);
}

int linear_int8_mixed_fp16_weights(const uint16_t* X, int64_t M, int64_t K, const uint16_t* W,
                                   int64_t N, int8_t* Wq, float* sw, int quantize_weight,
                                   const uint16_t* bias, float threshold, uint16_t* Y,
                                   void* workspace, size_t workspace_bytes,
                                   i8mm_stream_t stream) {
  const char* fn = "linear_int8_mixed_fp16_weights";
  I8MM_TRY(check_ptr(fn, "W", W, N * K > 0));
  return run_layer(fn, X, M, K, Wq, sw, N, bias, threshold, Y, workspace, workspace_bytes,
                   (hipStream_t)stream, W, quantize_weight != 0);
}

int outlier_detect_quantize(const uint16_t* X, int64_t M, int64_t K, float threshold,
                            void* workspace, size_t workspace_bytes, i8mm_stream_t stream) {
  const char* fn = "outlier_detect_quantize";
  I8MM_TRY(check_dims(fn, M, 0, K));
  if (std::isnan(threshold)) return fail(I8MM_EINVAL, "%s: threshold is NaN", fn);
  I8MM_TRY(check_ptr(fn, "X", X, M * K > 0));
  int64_t off[7], off_part = 0, off_kbl = 0;
  layout(M, K, off, &off_part, &off_kbl);
  I8MM_TRY(check_workspace(fn, workspace, workspace_bytes, off));
  if (M == 0) return ok();
  I8MM_TRY(check_device());
  I8MM_TRY(x_side(fn, X, M, K, i8mm::fp16_threshold_pattern(threshold),
                  static_cast<char*>(workspace), off, off_part, off_kbl, (hipStream_t)stream));
  return ok();
}

}  // extern "C"

namespace {

// Workspace of linear_int8_mixed_noalloc, for callers that cannot allocate:
// one copy per GPU the library runs on, held until the process ends. In host
// code `scratch` names a host-side stand-in, never the device memory: the
// device address comes from hipGetSymbolAddress, once per device.
static __device__ __align__(256) unsigned char scratch[I8MM_NOALLOC_SCRATCH_BYTES];

std::atomic<void*> g_scratch[kMaxDevices];

// Device address of `scratch` on the current device, looked up on the first
// call there (concurrent first calls look up the same address).
int scratch_address(const char* fn, void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(I8MM_ENODEVICE, "%s: no HIP device: %s", fn, hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices)
    return fail(I8MM_ENODEVICE, "%s: device %d beyond the %d the library tracks", fn, dev,
                kMaxDevices);
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (!p) {
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p)
      return fail(I8MM_ELAUNCH, "%s: hipGetSymbolAddress(scratch): %s", fn, hipGetErrorString(e));
    g_scratch[dev].store(p, std::memory_order_release);
  }
  *out = p;
  return I8MM_OK;
}

}  // namespace

extern "C" {

int linear_int8_mixed_noalloc(const uint16_t* X, int64_t M, int64_t K, const int8_t* Wq,
                              const float* sw, int64_t N, const uint16_t* bias, float threshold,
                              uint16_t* Y, i8mm_stream_t stream) {
  const char* fn = "linear_int8_mixed_noalloc";
  I8MM_TRY(check_layer_args(fn, X, M, K, Wq, sw, N, bias, threshold, Y));
  int64_t off[7];
  layout(M, K, off);
  if (off[6] > (int64_t)I8MM_NOALLOC_SCRATCH_BYTES)
    return fail(I8MM_EWORKSPACE,
                "%s: M=%lld, K=%lld need %lld bytes of workspace, more than the %lld of the "
                "library's scratch; use linear_int8_mixed with a workspace",
                fn, (long long)M, (long long)K, (long long)off[6],
                (long long)I8MM_NOALLOC_SCRATCH_BYTES);
  if (M == 0 || N == 0) return ok();
  I8MM_TRY(check_device());
  void* ws = nullptr;
  I8MM_TRY(scratch_address(fn, &ws));
  return run_layer(fn, X, M, K, Wq, sw, N, bias, threshold, Y, ws,
                   (size_t)I8MM_NOALLOC_SCRATCH_BYTES, (hipStream_t)stream, nullptr, false);
}

int i8mm_gelu_f16(const uint16_t* X, int64_t count, uint16_t* Y, i8mm_stream_t stream) {
  const char* fn = "i8mm_gelu_f16";
  if (count < 0) return fail(I8MM_EINVAL, "%s: negative count", fn);
  I8MM_TRY(check_ptr(fn, "X", X, count > 0));
  I8MM_TRY(check_ptr(fn, "Y", Y, count > 0));
  if (count == 0) return ok();
  I8MM_TRY(check_device());
  I8MM_TRY(launched(i8mm::launch_gelu(X, count, Y, (hipStream_t)stream), fn));
  return ok();
}

}  // extern "C"

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes of a cache and a batch, checked and narrowed into *a (pointers not
// looked at).
int cache_sizes(const char* fn, const i8mm_kv_cache* c, i8mm::KvArgs* a) {
  if (c->num_pages < 0 || c->page_tokens <= 0 || c->page_tokens > 65536 || c->kv_heads <= 0)
    return fail(I8MM_EINVAL, "%s: cache of %lld pages of %lld tokens, %lld heads", fn,
                (long long)c->num_pages, (long long)c->page_tokens, (long long)c->kv_heads);
  if (c->page_tokens % I8MM_KV_BLOCK != 0)
    return fail(I8MM_EALIGN, "%s: page_tokens=%lld is not a multiple of %d", fn,
                (long long)c->page_tokens, I8MM_KV_BLOCK);
  if (!i8mm::kv_head_dim_ok(c->head_dim))
    return fail(I8MM_EINVAL, "%s: head_dim=%lld is none of 64, 80, 96, 128, 256", fn,
                (long long)c->head_dim);
  const int64_t slots = c->page_tokens / I8MM_KV_BLOCK;
  // blocks are numbered in int32; heads and sequences are grid dimensions
  if (c->kv_heads > 65535 || slots > INT32_MAX / c->kv_heads ||
      c->num_pages > INT32_MAX / (slots * c->kv_heads))
    return fail(I8MM_EINVAL, "%s: more than 2^31 - 1 blocks or 65535 heads", fn);
  a->num_pages = (int)c->num_pages;
  a->slots = (int)slots;
  a->kv_heads = (int)c->kv_heads;
  a->head_dim = (int)c->head_dim;
  return I8MM_OK;
}

int kv_sizes(const char* fn, const i8mm_kv_cache* c, const i8mm_kv_batch* b, i8mm::KvArgs* a) {
  if (!c || !b) return fail(I8MM_EINVAL, "%s: cache or batch is NULL", fn);
  I8MM_TRY(cache_sizes(fn, c, a));
  if (b->num_seqs < 0 || b->max_pages < 0 || b->total_tokens < 0 || b->max_tokens < 0 ||
      b->max_len < 0)
    return fail(I8MM_EINVAL, "%s: negative size in the batch", fn);
  if (b->num_seqs > 65535 || b->total_tokens > INT32_MAX || b->max_tokens > INT32_MAX / 4 ||
      b->max_pages > INT32_MAX)
    return fail(I8MM_EINVAL, "%s: more than 65535 sequences or a size beyond int32", fn);
  if (!b->cu_tokens && b->total_tokens != b->num_seqs)
    return fail(I8MM_EINVAL, "%s: no cu_tokens, but %lld tokens for %lld sequences", fn,
                (long long)b->total_tokens, (long long)b->num_seqs);
  const int64_t room = b->max_pages * c->page_tokens;
  // (no pages: every token is absent, as in sequences of length 0)
  const int64_t cap = c->num_pages > 0 ? std::min(b->max_len, room) : 0;
  if (cap > INT32_MAX / 2) return fail(I8MM_EINVAL, "%s: max_len beyond 2^30 tokens", fn);
  a->num_seqs = (int)b->num_seqs;
  a->max_pages = (int)b->max_pages;
  a->total_tokens = (int)b->total_tokens;
  a->max_tokens = (int)std::min(b->max_tokens, b->cu_tokens ? b->total_tokens : (int64_t)1);
  a->len_cap = (int)cap;
  return I8MM_OK;
}

int cache_pointers(const char* fn, const i8mm_kv_cache* c, i8mm::KvArgs* a) {
  const bool some = c->num_pages > 0;
  I8MM_TRY(check_ptr(fn, "k_codes", c->k_codes, some));
  I8MM_TRY(check_ptr(fn, "k_absmax", c->k_absmax, some));
  I8MM_TRY(check_ptr(fn, "v_codes", c->v_codes, some));
  I8MM_TRY(check_ptr(fn, "v_absmax", c->v_absmax, some));
  a->k_codes = c->k_codes;
  a->k_absmax = c->k_absmax;
  a->v_codes = c->v_codes;
  a->v_absmax = c->v_absmax;
  return I8MM_OK;
}

int kv_check(const char* fn, const i8mm_kv_cache* c, const i8mm_kv_batch* b, i8mm::KvArgs* a) {
  I8MM_TRY(kv_sizes(fn, c, b, a));
  I8MM_TRY(cache_pointers(fn, c, a));
  if (!b->page_table && b->num_seqs * b->max_pages > 0)
    return fail(I8MM_EINVAL, "%s: page_table is NULL", fn);
  if (!b->seq_lens && b->num_seqs > 0) return fail(I8MM_EINVAL, "%s: seq_lens is NULL", fn);
  if (!aligned4(b->page_table) || !aligned4(b->seq_lens) || !aligned4(b->cu_tokens))
    return fail(I8MM_EALIGN, "%s: page_table, seq_lens or cu_tokens is not 4-byte aligned", fn);
  a->page_table = b->page_table;
  a->seq_lens = b->seq_lens;
  a->cu_tokens = b->cu_tokens;
  return I8MM_OK;
}

int rotary_check(const char* fn, const i8mm_rotary* r, const i8mm::KvArgs& a,
                 i8mm::RotaryArgs* out) {
  *out = i8mm::RotaryArgs{nullptr, nullptr, 0, 0};
  if (!r) return I8MM_OK;
  if (r->dim <= 0 || r->dim % 16 != 0 || r->dim > a.head_dim)
    return fail(I8MM_EINVAL, "%s: rotary dim=%lld is not a multiple of 16 up to %d", fn,
                (long long)r->dim, a.head_dim);
  if (r->positions < a.len_cap)
    return fail(I8MM_EINVAL, "%s: rotary tables of %lld positions, sequences up to %d", fn,
                (long long)r->positions, a.len_cap);
  I8MM_TRY(check_ptr(fn, "cos", r->cos, a.len_cap > 0));
  I8MM_TRY(check_ptr(fn, "sin", r->sin, a.len_cap > 0));
  if (a.len_cap == 0) return I8MM_OK;   // no token has a position: the tables may be empty
  *out = i8mm::RotaryArgs{r->cos, r->sin, (int)r->dim, r->interleaved != 0};
  return I8MM_OK;
}

// The queries that share a key/value head are rows, numbered in int32, those of
// a sequence up to half of it; the rows of all heads are few enough for the
// workspace's bytes to stay in 64 bits.
bool heads_ok(const i8mm::KvArgs& a, int64_t q_heads) {
  return q_heads > 0 && q_heads <= 65535 && q_heads % a.kv_heads == 0 &&
         a.max_tokens <= INT32_MAX / 2 / (q_heads / a.kv_heads) &&
         a.total_tokens <= (INT32_MAX - 65536) / (q_heads / a.kv_heads) &&
         a.total_tokens <= (int64_t{1} << 40) / q_heads;
}

int heads_check(const char* fn, const i8mm::KvArgs& a, int64_t q_heads) {
  if (heads_ok(a, q_heads)) return I8MM_OK;
  return fail(I8MM_EINVAL, "%s: q_heads=%lld is not a multiple of %d key/value heads, or too many "
              "for %d tokens, %d a sequence", fn, (long long)q_heads, a.kv_heads, a.total_tokens,
              a.max_tokens);
}

// No row of the packed tensors belongs to a sequence.
bool no_tokens(const i8mm::KvArgs& a) {
  return a.total_tokens == 0 || a.max_tokens == 0 || a.num_seqs == 0;
}

// All rows of an output, where none belongs to a sequence.
int zero_halfs(const char* fn, uint16_t* p, int64_t count, i8mm_stream_t stream) {
  return launched(i8mm::launch_fill_u32(reinterpret_cast<uint32_t*>(p), count / 2, 0u,
                                        (hipStream_t)stream), fn);
}

// 16-byte loads of 8 halfs at any token and head.
int strides_check(const char* fn, const char* name, const void* p, bool required, int64_t ts,
                  int64_t hs) {
  I8MM_TRY(check_ptr(fn, name, p, required));
  if (ts < 0 || hs < 0) return fail(I8MM_EINVAL, "%s: negative stride of %s", fn, name);
  if (ts % 8 != 0 || hs % 8 != 0)
    return fail(I8MM_EALIGN, "%s: strides of %s are not multiples of 8 elements", fn, name);
  return I8MM_OK;
}

}  // namespace

extern "C" {

int int8_kv_cache_append(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride,
                         const uint16_t* v, int64_t v_token_stride, int64_t v_head_stride,
                         const i8mm_kv_cache* cache, const i8mm_kv_batch* batch,
                         const i8mm_rotary* rotary, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_append";
  i8mm::KvArgs a;
  i8mm::RotaryArgs r;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(rotary_check(fn, rotary, a, &r));
  I8MM_TRY(strides_check(fn, "k", k, a.total_tokens > 0, k_token_stride, k_head_stride));
  I8MM_TRY(strides_check(fn, "v", v, a.total_tokens > 0, v_token_stride, v_head_stride));
  if (no_tokens(a) || a.len_cap == 0 || a.num_pages == 0) return ok();
  I8MM_TRY(check_device());
  I8MM_TRY(launched(i8mm::launch_kv_append(k, k_token_stride, k_head_stride, v, v_token_stride,
                                           v_head_stride, a, r, (hipStream_t)stream),
                    fn));
  return ok();
}

int int8_kv_cache_read(const i8mm_kv_cache* cache, const i8mm_kv_batch* batch, uint16_t* k,
                       uint16_t* v, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_read";
  i8mm::KvArgs a;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(check_ptr(fn, "k", k, false));
  I8MM_TRY(check_ptr(fn, "v", v, false));
  if ((!k && !v) || a.total_tokens == 0) return ok();
  I8MM_TRY(check_device());
  if (no_tokens(a)) {
    if (k) I8MM_TRY(zero_halfs(fn, k, (int64_t)a.total_tokens * a.kv_heads * a.head_dim, stream));
    if (v) I8MM_TRY(zero_halfs(fn, v, (int64_t)a.total_tokens * a.kv_heads * a.head_dim, stream));
    return ok();
  }
  I8MM_TRY(launched(i8mm::launch_kv_read(a, k, v, (hipStream_t)stream), fn));
  return ok();
}

size_t int8_kv_cache_attention_workspace_bytes(const i8mm_kv_cache* cache,
                                               const i8mm_kv_batch* batch, int64_t q_heads) {
  i8mm::KvArgs a;
  if (kv_sizes("int8_kv_cache_attention_workspace_bytes", cache, batch, &a) != I8MM_OK) return 0;
  if (!heads_ok(a, q_heads)) return 0;
  return i8mm::attn_workspace_bytes(a, (int)q_heads);
}

int int8_kv_cache_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                            int64_t q_heads, const i8mm_kv_cache* cache,
                            const i8mm_kv_batch* batch, const i8mm_rotary* rotary, float scale,
                            int causal, int64_t window, const float* alibi_slopes, uint16_t* out,
                            void* workspace, size_t workspace_bytes, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_attention";
  i8mm::KvArgs a;
  i8mm::RotaryArgs r;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(rotary_check(fn, rotary, a, &r));
  I8MM_TRY(heads_check(fn, a, q_heads));
  I8MM_TRY(strides_check(fn, "q", q, a.total_tokens > 0, q_token_stride, q_head_stride));
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(I8MM_EINVAL, "%s: scale is not finite and positive", fn);
  if (causal != 0 && causal != 1) return fail(I8MM_EINVAL, "%s: causal is not 0 or 1", fn);
  if (window < 0 || (window > 0 && !causal))
    return fail(I8MM_EINVAL, "%s: window is negative, or given without causal", fn);
  if (!aligned4(alibi_slopes))
    return fail(I8MM_EALIGN, "%s: alibi_slopes is not 4-byte aligned", fn);
  I8MM_TRY(check_ptr(fn, "out", out, a.total_tokens > 0));
  const size_t need = i8mm::attn_workspace_bytes(a, (int)q_heads);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(I8MM_EWORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn,
                  workspace ? workspace_bytes : (size_t)0, need);
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
      return fail(I8MM_EALIGN, "%s: workspace is not 256-byte aligned", fn);
  }
  if (a.total_tokens == 0) return ok();
  I8MM_TRY(check_device());
  if (no_tokens(a)) {
    I8MM_TRY(zero_halfs(fn, out, a.total_tokens * q_heads * a.head_dim, stream));
    return ok();
  }
  i8mm::AttnArgs t;
  t.q = q;
  t.q_ts = q_token_stride;
  t.q_hs = q_head_stride;
  t.slopes = alibi_slopes;
  t.out = out;
  t.part = static_cast<float*>(workspace);
  t.scale_log2 = scale * 1.44269504088896340736f;
  t.q_heads = (int)q_heads;
  t.causal = causal;
  t.window = (int)std::min<int64_t>(window, INT32_MAX / 2);
  I8MM_TRY(launched(i8mm::launch_kv_attention(a, r, t, (hipStream_t)stream), fn));
  return ok();
}

}  // extern "C"

namespace {

// Arrays in words of 32 bits, and whether any that is written (a workspace among them)
// shares memory with one that is read or with another that is written.
struct Words32 {
  const void* p;
  int64_t n;
};
bool overlap(const Words32& x, const Words32& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && x.n > 0 && y.n > 0 && a < b + 4 * (uintptr_t)y.n && b < a + 4 * (uintptr_t)x.n;
}
int check_apart(const char* fn, std::initializer_list<Words32> written,
                std::initializer_list<Words32> read) {
  for (const Words32* w = written.begin(); w != written.end(); ++w) {
    bool shared = false;
    for (const Words32& r : read) shared = shared || overlap(*w, r);
    for (const Words32* o = w + 1; o != written.end(); ++o) shared = shared || overlap(*w, *o);
    if (shared)
      return fail(I8MM_EINVAL, "%s: an output or the workspace overlaps an input or another output", fn);
  }
  return I8MM_OK;
}

int beam_sizes(const char* fn, int fp32, int64_t batch, int64_t beams, int64_t vocab,
               int64_t count, i8mm::BeamArgs* a) {
  if (fp32 != 0 && fp32 != 1) return fail(I8MM_EINVAL, "%s: logits_fp32 is not 0 or 1", fn);
  if (batch < 0 || beams < 0 || vocab < 0)
    return fail(I8MM_EINVAL, "%s: negative size", fn);
  // (rows are numbered in int32, and blocks of up to 65536 words of them launched)
  if (beams > I8MM_MAX_BEAMS || vocab > I8MM_MAX_VOCAB ||
      batch > (1 << 23) / std::max<int64_t>(beams, 1) / (vocab / 65536 + 1))
    return fail(I8MM_EINVAL, "%s: more than %d beams, %d words or 2^23 rows of 65536 words", fn,
                I8MM_MAX_BEAMS, I8MM_MAX_VOCAB);
  if (count < 1 || count > I8MM_MAX_BEAM_COUNT)
    return fail(I8MM_EINVAL, "%s: count=%lld is not 1 .. %d", fn, (long long)count,
                I8MM_MAX_BEAM_COUNT);
  a->fp32 = fp32;
  a->batch = (int)batch;
  a->beams = (int)beams;
  a->vocab = vocab;
  a->count = (int)count;
  return I8MM_OK;
}

int check_ints(const char* fn, const char* name, const void* p, bool required) {
  if (!p && required) return fail(I8MM_EINVAL, "%s: %s is NULL", fn, name);
  if (!aligned4(p)) return fail(I8MM_EALIGN, "%s: %s is not 4-byte aligned", fn, name);
  return I8MM_OK;
}

int check_scratch(const char* fn, const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return I8MM_OK;
  if (!workspace || bytes < need)
    return fail(I8MM_EWORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn,
                workspace ? bytes : (size_t)0, need);
  if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return fail(I8MM_EALIGN, "%s: workspace is not 256-byte aligned", fn);
  return I8MM_OK;
}

}  // namespace

extern "C" {

size_t i8mm_beam_select_workspace_bytes(int logits_fp32, int64_t batch, int64_t beams,
                                        int64_t vocab, int64_t count) {
  i8mm::BeamArgs a;
  if (beam_sizes("i8mm_beam_select_workspace_bytes", logits_fp32, batch, beams, vocab, count, &a) !=
      I8MM_OK)
    return 0;
  return batch == 0 ? 0 : i8mm::beam_workspace_bytes(a);
}

int i8mm_beam_select(const void* logits, int logits_fp32, int64_t row_stride, const float* scores,
                     const int32_t* live, int64_t batch, int64_t beams, int64_t vocab,
                     int64_t count, int32_t eos, float* out_scores, int32_t* out_tokens,
                     int32_t* out_parents, int32_t* out_live, void* workspace,
                     size_t workspace_bytes, i8mm_stream_t stream) {
  const char* fn = "i8mm_beam_select";
  i8mm::BeamArgs a;
  I8MM_TRY(beam_sizes(fn, logits_fp32, batch, beams, vocab, count, &a));
  const int64_t rows = batch * beams;
  if (row_stride < vocab)
    return fail(I8MM_EINVAL, "%s: row_stride=%lld is less than vocab=%lld", fn,
                (long long)row_stride, (long long)vocab);
  if (rows > 0 && row_stride > INT64_MAX / 8 / rows)
    return fail(I8MM_EINVAL, "%s: rows beyond 64 bits", fn);
  if (eos < -1 || (eos >= 0 && eos >= vocab))
    return fail(I8MM_EINVAL, "%s: eos=%d is neither -1 nor one of %lld words", fn, eos,
                (long long)vocab);
  if (!logits && rows > 0 && vocab > 0) return fail(I8MM_EINVAL, "%s: logits is NULL", fn);
  if (reinterpret_cast<uintptr_t>(logits) % (logits_fp32 ? 4 : 2) != 0)
    return fail(I8MM_EALIGN, "%s: logits is not aligned to its elements", fn);
  I8MM_TRY(check_ints(fn, "scores", scores, rows > 0));
  I8MM_TRY(check_ints(fn, "live", live, false));
  I8MM_TRY(check_ints(fn, "out_scores", out_scores, batch > 0));
  I8MM_TRY(check_ints(fn, "out_tokens", out_tokens, batch > 0));
  I8MM_TRY(check_ints(fn, "out_parents", out_parents, batch > 0));
  I8MM_TRY(check_ints(fn, "out_live", out_live, batch > 0));
  const size_t need = batch == 0 ? 0 : i8mm::beam_workspace_bytes(a);
  I8MM_TRY(check_scratch(fn, workspace, workspace_bytes, need));
  // (from the first row's first word to the last row's last)
  const int64_t span = rows > 0 ? (rows - 1) * row_stride + vocab : 0;
  I8MM_TRY(check_apart(fn, {{out_scores, batch * count}, {out_tokens, batch * count},
                            {out_parents, batch * count}, {out_live, batch * count},
                            {workspace, (int64_t)(need / 4)}},
                       {{scores, rows}, {live, rows}, {logits, logits_fp32 ? span : (span + 1) / 2}}));
  if (batch == 0) return ok();
  I8MM_TRY(check_device());
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.live = live;
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  a.out_live = out_live;
  a.ws = workspace;
  a.eos = eos;
  I8MM_TRY(launched(i8mm::launch_beam_select(a, (hipStream_t)stream), fn));
  return ok();
}

}  // extern "C"

namespace {

// Sizes of the calls on page tables, narrowed into *a.
int pages_sizes(const char* fn, int64_t num_seqs, int64_t max_pages, int64_t num_rows,
                int64_t num_pages, int64_t page_tokens, i8mm::PagesArgs* a) {
  *a = i8mm::PagesArgs{};
  if (num_seqs < 0 || max_pages < 0 || num_rows < 0 || num_pages < 0)
    return fail(I8MM_EINVAL, "%s: negative size", fn);
  if (page_tokens <= 0 || page_tokens > 65536)
    return fail(I8MM_EINVAL, "%s: pages of %lld tokens", fn, (long long)page_tokens);
  if (page_tokens % I8MM_KV_BLOCK != 0)
    return fail(I8MM_EALIGN, "%s: page_tokens=%lld is not a multiple of %d", fn,
                (long long)page_tokens, I8MM_KV_BLOCK);
  if (num_seqs > 65535 || num_rows > 65535 || num_pages > INT32_MAX - 8192 ||
      max_pages > (1 << 30) / page_tokens ||
      std::max(num_seqs, num_rows) * (max_pages + 1) > INT32_MAX)
    return fail(I8MM_EINVAL, "%s: more than 65535 sequences, 2^30 tokens of one or 2^31 pages", fn);
  a->num_seqs = (int)num_seqs;
  a->max_pages = (int)max_pages;
  a->num_rows = (int)num_rows;
  a->num_pages = (int)num_pages;
  a->page_tokens = (int)page_tokens;
  return I8MM_OK;
}

}  // namespace

extern "C" {

size_t i8mm_kv_pages_workspace_bytes(int64_t num_rows, int64_t max_pages, int64_t num_pages) {
  i8mm::PagesArgs a;
  if (pages_sizes("i8mm_kv_pages_workspace_bytes", 0, max_pages, num_rows, num_pages, I8MM_KV_BLOCK,
                  &a) != I8MM_OK)
    return 0;
  return i8mm::kv_pages_workspace_bytes(a, a.num_rows);
}

}  // extern "C"

namespace {

// A step of the page tables; batch_lens and full are there or not together.
int pages_step(const char* fn, const int32_t* page_table, const int32_t* seq_lens, int64_t num_seqs,
               int64_t max_pages, const int32_t* parents, const int32_t* keep,
               const int32_t* new_tokens, int64_t new_all, int64_t num_rows, int64_t num_pages,
               int64_t page_tokens, int64_t max_len, bool batch, int32_t* out_table,
               int32_t* out_lens, int32_t* batch_lens, int32_t* full, int32_t* copies,
               int32_t* counts, void* workspace, size_t workspace_bytes, i8mm_stream_t stream) {
  i8mm::PagesArgs a;
  I8MM_TRY(pages_sizes(fn, num_seqs, max_pages, num_rows, num_pages, page_tokens, &a));
  if (new_all < 0 || new_all > (1 << 30))
    return fail(I8MM_EINVAL, "%s: %lld new tokens", fn, (long long)new_all);
  if (max_len < 0) return fail(I8MM_EINVAL, "%s: max_len=%lld", fn, (long long)max_len);
  I8MM_TRY(check_ints(fn, "page_table", page_table, num_seqs * max_pages > 0));
  I8MM_TRY(check_ints(fn, "seq_lens", seq_lens, num_seqs > 0));
  I8MM_TRY(check_ints(fn, "parents", parents, num_rows > 0));
  I8MM_TRY(check_ints(fn, "keep", keep, false));
  I8MM_TRY(check_ints(fn, "new_tokens", new_tokens, false));
  I8MM_TRY(check_ints(fn, "out_table", out_table, num_rows * max_pages > 0));
  I8MM_TRY(check_ints(fn, "out_lens", out_lens, num_rows > 0));
  I8MM_TRY(check_ints(fn, "batch_lens", batch_lens, batch && num_rows > 0));
  I8MM_TRY(check_ints(fn, "full", full, batch));
  I8MM_TRY(check_ints(fn, "copies", copies, num_rows > 0));
  I8MM_TRY(check_ints(fn, "counts", counts, true));
  const size_t need = i8mm::kv_pages_workspace_bytes(a, a.num_rows);
  I8MM_TRY(check_scratch(fn, workspace, workspace_bytes, need));
  I8MM_TRY(check_apart(fn, {{out_table, num_rows * max_pages}, {out_lens, num_rows},
                            {batch_lens, num_rows}, {full, 1}, {copies, 3 * num_rows}, {counts, 2},
                            {workspace, (int64_t)(need / 4)}},
                       {{page_table, num_seqs * max_pages}, {seq_lens, num_seqs}, {parents, num_rows},
                        {keep, num_rows}, {new_tokens, num_rows}}));
  I8MM_TRY(check_device());
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.keep = keep;
  a.new_tokens = new_tokens;
  a.new_all = (int)new_all;
  a.out_table = out_table;
  a.out_lens = out_lens;
  a.batch_lens = batch_lens;
  a.full = full;
  a.max_len = (int)std::min<int64_t>(max_len, INT32_MAX);
  a.copies = copies;
  a.counts = counts;
  I8MM_TRY(launched(i8mm::launch_kv_pages_step(a, workspace, (hipStream_t)stream), fn));
  return ok();
}

}  // namespace

extern "C" {

int i8mm_kv_pages_step(const int32_t* page_table, const int32_t* seq_lens, int64_t num_seqs,
                       int64_t max_pages, const int32_t* parents, const int32_t* keep,
                       const int32_t* new_tokens, int64_t new_all, int64_t num_rows,
                       int64_t num_pages, int64_t page_tokens, int32_t* out_table,
                       int32_t* out_lens, int32_t* copies, int32_t* counts, void* workspace,
                       size_t workspace_bytes, i8mm_stream_t stream) {
  return pages_step("i8mm_kv_pages_step", page_table, seq_lens, num_seqs, max_pages, parents, keep,
                    new_tokens, new_all, num_rows, num_pages, page_tokens, INT32_MAX, false, out_table,
                    out_lens, nullptr, nullptr, copies, counts, workspace, workspace_bytes, stream);
}

int i8mm_kv_pages_step_batch(const int32_t* page_table, const int32_t* seq_lens, int64_t num_seqs,
                             int64_t max_pages, const int32_t* parents, const int32_t* keep,
                             const int32_t* new_tokens, int64_t new_all, int64_t num_rows,
                             int64_t num_pages, int64_t page_tokens, int64_t max_len,
                             int32_t* out_table, int32_t* out_lens, int32_t* batch_lens,
                             int32_t* full, int32_t* copies, int32_t* counts, void* workspace,
                             size_t workspace_bytes, i8mm_stream_t stream) {
  return pages_step("i8mm_kv_pages_step_batch", page_table, seq_lens, num_seqs, max_pages, parents,
                    keep, new_tokens, new_all, num_rows, num_pages, page_tokens, max_len, true,
                    out_table, out_lens, batch_lens, full, copies, counts, workspace, workspace_bytes,
                    stream);
}

int i8mm_kv_pages_compact(const int32_t* page_table, const int32_t* seq_lens, int64_t num_seqs,
                          int64_t max_pages, int64_t num_pages, int64_t page_tokens,
                          int32_t* out_table, int32_t* copies, int32_t* counts, void* workspace,
                          size_t workspace_bytes, i8mm_stream_t stream) {
  const char* fn = "i8mm_kv_pages_compact";
  i8mm::PagesArgs a;
  I8MM_TRY(pages_sizes(fn, num_seqs, max_pages, 0, num_pages, page_tokens, &a));
  const int64_t entries = num_seqs * max_pages;
  I8MM_TRY(check_ints(fn, "page_table", page_table, entries > 0));
  I8MM_TRY(check_ints(fn, "seq_lens", seq_lens, num_seqs > 0));
  I8MM_TRY(check_ints(fn, "out_table", out_table, entries > 0));
  I8MM_TRY(check_ints(fn, "copies", copies, num_pages >= 2));
  I8MM_TRY(check_ints(fn, "counts", counts, true));
  const size_t need = i8mm::kv_pages_workspace_bytes(a, a.num_seqs);
  I8MM_TRY(check_scratch(fn, workspace, workspace_bytes, need));
  // (a table is renamed entry by entry, in place too)
  I8MM_TRY(check_apart(fn, {{out_table, entries}, {copies, num_pages / 2 * 3}, {counts, 2},
                            {workspace, (int64_t)(need / 4)}},
                       {{out_table == page_table ? nullptr : page_table, entries},
                        {seq_lens, num_seqs}}));
  I8MM_TRY(check_device());
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out_table = out_table;
  a.copies = copies;
  a.counts = counts;
  I8MM_TRY(launched(i8mm::launch_kv_pages_compact(a, workspace, (hipStream_t)stream), fn));
  return ok();
}

int int8_kv_cache_copy_pages(const i8mm_kv_cache* cache, uint16_t* k_means, const int32_t* copies,
                             const int32_t* count, int64_t max_copies, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_copy_pages";
  i8mm::KvArgs a = {};
  if (!cache) return fail(I8MM_EINVAL, "%s: cache is NULL", fn);
  I8MM_TRY(cache_sizes(fn, cache, &a));
  I8MM_TRY(cache_pointers(fn, cache, &a));
  I8MM_TRY(check_ptr(fn, "k_means", k_means, false));
  if (max_copies < 0 || max_copies > INT32_MAX)
    return fail(I8MM_EINVAL, "%s: %lld copies", fn, (long long)max_copies);
  I8MM_TRY(check_ints(fn, "copies", copies, max_copies > 0));
  I8MM_TRY(check_ints(fn, "count", count, max_copies > 0));
  if (max_copies == 0 || a.num_pages == 0) return ok();
  I8MM_TRY(check_device());
  I8MM_TRY(launched(i8mm::launch_kv_copy_pages(a, k_means, copies, count, (int)max_copies,
                                               (hipStream_t)stream), fn));
  return ok();
}

}  // extern "C"

namespace {

// A list of pages for each token and head.
int count_check(const char* fn, const i8mm::KvArgs& a, int64_t count) {
  if (count < 1 || count > (1 << 30) / (a.slots * I8MM_KV_BLOCK))
    return fail(I8MM_EINVAL, "%s: lists of %lld pages of %d tokens", fn, (long long)count,
                a.slots * I8MM_KV_BLOCK);
  return I8MM_OK;
}

}  // namespace

extern "C" {

int int8_kv_cache_page_means(const i8mm_kv_cache* cache, const i8mm_kv_batch* batch,
                             uint16_t* k_means, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_page_means";
  i8mm::KvArgs a;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(check_ptr(fn, "k_means", k_means, a.num_pages > 0));
  if (no_tokens(a) || a.len_cap == 0) return ok();
  if ((i8mm::page_means_tasks(a) + 3) / 4 > i8mm::max_grid(256))
    return fail(I8MM_EINVAL, "%s: %d new tokens of a sequence touch too many pages of %d heads", fn,
                a.max_tokens, a.kv_heads);
  I8MM_TRY(check_device());
  I8MM_TRY(launched(i8mm::launch_kv_page_means(a, k_means, (hipStream_t)stream), fn));
  return ok();
}

int int8_kv_cache_select_pages(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t q_heads, const i8mm_kv_cache* cache, const uint16_t* k_means,
                               const i8mm_kv_batch* batch, const i8mm_rotary* rotary, int64_t count,
                               int64_t first, int64_t recent, int32_t* pages, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_select_pages";
  i8mm::KvArgs a;
  i8mm::RotaryArgs r;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(rotary_check(fn, rotary, a, &r));
  I8MM_TRY(heads_check(fn, a, q_heads));
  I8MM_TRY(strides_check(fn, "q", q, a.total_tokens > 0, q_token_stride, q_head_stride));
  I8MM_TRY(check_ptr(fn, "k_means", k_means, a.num_pages > 0));
  I8MM_TRY(count_check(fn, a, count));
  if (first < 0 || recent < 1 || first > count || recent > count - first)
    return fail(I8MM_EINVAL, "%s: first=%lld and recent=%lld of count=%lld", fn, (long long)first,
                (long long)recent, (long long)count);
  const int64_t page_tokens = (int64_t)a.slots * I8MM_KV_BLOCK;
  if ((a.len_cap + page_tokens - 1) / page_tokens - first - recent > I8MM_MAX_SELECT_PAGES)
    return fail(I8MM_EINVAL, "%s: more than %d pages to choose from in %d tokens", fn,
                I8MM_MAX_SELECT_PAGES, a.len_cap);
  if (!no_tokens(a) && (int64_t)a.total_tokens * a.kv_heads > i8mm::max_grid(256))
    return fail(I8MM_EINVAL, "%s: %d tokens of %d heads are more than 2^24 - 1 lists", fn,
                a.total_tokens, a.kv_heads);
  I8MM_TRY(check_ints(fn, "pages", pages, a.total_tokens > 0));
  if (a.total_tokens == 0) return ok();
  I8MM_TRY(check_device());
  if (no_tokens(a)) {
    I8MM_TRY(launched(i8mm::launch_fill_u32(reinterpret_cast<uint32_t*>(pages),
                                            (int64_t)a.total_tokens * a.kv_heads * count, ~0u,
                                            (hipStream_t)stream), fn));
    return ok();
  }
  I8MM_TRY(launched(i8mm::launch_kv_select_pages(a, r, q, q_token_stride, q_head_stride, (int)q_heads,
                                                 k_means, (int)count, (int)first, (int)recent, pages,
                                                 (hipStream_t)stream), fn));
  return ok();
}

size_t int8_kv_cache_attention_pages_workspace_bytes(const i8mm_kv_cache* cache,
                                                     const i8mm_kv_batch* batch, int64_t q_heads,
                                                     int64_t count) {
  const char* fn = "int8_kv_cache_attention_pages_workspace_bytes";
  i8mm::KvArgs a;
  if (kv_sizes(fn, cache, batch, &a) != I8MM_OK || !heads_ok(a, q_heads) ||
      count_check(fn, a, count) != I8MM_OK)
    return 0;
  return i8mm::attn_pages_workspace_bytes(a, (int)q_heads, (int)count);
}

int int8_kv_cache_attention_pages(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                  int64_t q_heads, const i8mm_kv_cache* cache,
                                  const i8mm_kv_batch* batch, const i8mm_rotary* rotary,
                                  const int32_t* pages, int64_t count, float scale, uint16_t* out,
                                  void* workspace, size_t workspace_bytes, i8mm_stream_t stream) {
  const char* fn = "int8_kv_cache_attention_pages";
  i8mm::KvArgs a;
  i8mm::RotaryArgs r;
  I8MM_TRY(kv_check(fn, cache, batch, &a));
  I8MM_TRY(rotary_check(fn, rotary, a, &r));
  I8MM_TRY(heads_check(fn, a, q_heads));
  I8MM_TRY(strides_check(fn, "q", q, a.total_tokens > 0, q_token_stride, q_head_stride));
  I8MM_TRY(count_check(fn, a, count));
  I8MM_TRY(check_ints(fn, "pages", pages, a.total_tokens > 0));
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(I8MM_EINVAL, "%s: scale is not finite and positive", fn);
  I8MM_TRY(check_ptr(fn, "out", out, a.total_tokens > 0));
  if (!no_tokens(a) && a.len_cap > 0 && !i8mm::attn_pages_fits(a, (int)q_heads, (int)count))
    return fail(I8MM_EINVAL, "%s: too many lists, %d tokens of %d heads of %lld queries", fn,
                a.total_tokens, a.kv_heads, (long long)(q_heads / a.kv_heads));
  I8MM_TRY(check_scratch(fn, workspace, workspace_bytes,
                         i8mm::attn_pages_workspace_bytes(a, (int)q_heads, (int)count)));
  if (a.total_tokens == 0) return ok();
  I8MM_TRY(check_device());
  if (no_tokens(a) || a.len_cap == 0) {
    I8MM_TRY(zero_halfs(fn, out, a.total_tokens * q_heads * a.head_dim, stream));
    return ok();
  }
  i8mm::AttnArgs t = {};
  t.q = q;
  t.q_ts = q_token_stride;
  t.q_hs = q_head_stride;
  t.out = out;
  t.part = static_cast<float*>(workspace);
  t.scale_log2 = scale * 1.44269504088896340736f;
  t.q_heads = (int)q_heads;
  t.causal = 1;
  I8MM_TRY(launched(i8mm::launch_kv_attention_pages(a, r, t, pages, (int)count, (hipStream_t)stream),
                    fn));
  return ok();
}

}  // extern "C"
