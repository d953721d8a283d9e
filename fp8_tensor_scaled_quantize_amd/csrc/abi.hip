// C ABI of libfp8mi: argument validation, status reporting and dispatch to
// the kernel launchers.  Every check runs before any HIP call, so a rejected
// call has no side effects.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "../../include/fp8mi.h"
#include "fp8mi_internal.h"

namespace fp8mi {

static thread_local char g_err[512] = "";

static fp8mi_status fail(fp8mi_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

static fp8mi_status from_hip(hipError_t e, const char* where) {
  if (e == hipSuccess) return FP8MI_OK;
  return fail(FP8MI_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

int device_cu_count() {
  static std::mutex mu;
  static std::vector<int> cache;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  std::lock_guard<std::mutex> lock(mu);
  if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
  if (cache[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cache[dev] = n;
  }
  return cache[dev];
}

int env_int_in(const char* name, int lo, int hi, int dflt) {
  const char* e = getenv(name);
  if (!e || !*e) return dflt;
  char* end = nullptr;
  const long v = strtol(e, &end, 10);
  return (*end == '\0' && v >= lo && v <= hi) ? (int)v : dflt;
}

static_assert(kDynWorkspaceBytes == FP8MI_DYNAMIC_WORKSPACE_BYTES, "dynamic workspace size");
static_assert(kNormMaxCols == FP8MI_NORM_MAX_COLS, "norm column limit");

static bool valid_fmt(int f) { return f == FP8MI_E4M3 || f == FP8MI_E5M2; }
static bool valid_dtype(int d) { return d == FP8MI_F32 || d == FP8MI_F16 || d == FP8MI_BF16; }
static int dtype_bytes(int d) { return d == FP8MI_F32 ? 4 : 2; }

// rows x ld elements of elem bytes stay within 2^62 bytes: no allocation is
// that large, and the bound keeps every 64-bit index product in the kernels
// (and the checks below) from overflowing.
static bool span_ok(int64_t rows, int64_t ld, int64_t elem) {
  if (rows <= 0 || ld <= 0) return true;
  return ld <= (INT64_C(1) << 62) / elem / rows;
}

static fp8mi_status check_scale_ring(const float* scale, uint32_t* ring, int32_t H) {
  if ((scale == nullptr) == (ring == nullptr))
    return fail(FP8MI_ERR_ARG, "give exactly one of scale and ring (scale=%p ring=%p)", (const void*)scale,
                (void*)ring);
  if (ring) {
    if (H < 1 || H > FP8MI_MAX_HIST) return fail(FP8MI_ERR_SHAPE, "hist_len %d outside [1, %d]", H, FP8MI_MAX_HIST);
    if (reinterpret_cast<uintptr_t>(ring) & 3u) return fail(FP8MI_ERR_ARG, "ring must be 4-byte aligned");
  }
  return FP8MI_OK;
}

static fp8mi_status check_input(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x) {
  if (!valid_dtype(dt)) return fail(FP8MI_ERR_ENUM, "x_dtype %d is not FP8MI_F32/F16/BF16", dt);
  if (rows < 0 || cols < 0) return fail(FP8MI_ERR_SHAPE, "negative shape rows=%lld cols=%lld", (long long)rows,
                                        (long long)cols);
  if (rows > 0 && ld_x < cols) return fail(FP8MI_ERR_SHAPE, "ld_x %lld < cols %lld", (long long)ld_x, (long long)cols);
  if (!span_ok(rows, ld_x, dtype_bytes(dt)))
    return fail(FP8MI_ERR_SHAPE, "rows %lld x ld_x %lld beyond 2^62 bytes", (long long)rows, (long long)ld_x);
  if (rows > 0 && cols > 0 && x == nullptr) return fail(FP8MI_ERR_NULL, "x is NULL");
  if (reinterpret_cast<uintptr_t>(x) % dtype_bytes(dt)) return fail(FP8MI_ERR_ARG, "x not aligned to its element size");
  return FP8MI_OK;
}

// A further matrix of the norm calls (dtype dt, [rows, cols]): required, or
// NULL when it is optional.
static fp8mi_status check_matrix(const char* name, const void* m, bool required, int dt, int64_t rows, int64_t cols,
                                 int64_t ld) {
  if (!m) {
    if (required && rows > 0 && cols > 0) return fail(FP8MI_ERR_NULL, "%s is NULL", name);
    return FP8MI_OK;
  }
  if (rows > 0 && ld < cols)
    return fail(FP8MI_ERR_SHAPE, "leading dimension %lld of %s < cols %lld", (long long)ld, name, (long long)cols);
  if (!span_ok(rows, ld, dtype_bytes(dt)))
    return fail(FP8MI_ERR_SHAPE, "%s: rows %lld x ld %lld beyond 2^62 bytes", name, (long long)rows, (long long)ld);
  if (reinterpret_cast<uintptr_t>(m) % dtype_bytes(dt))
    return fail(FP8MI_ERR_ARG, "%s not aligned to its element size", name);
  return FP8MI_OK;
}

static fp8mi_status check_norm_weight(const void* weight, int dt, int64_t cols) {
  if (cols > kNormMaxCols)
    return fail(FP8MI_ERR_UNSUPPORTED, "cols %lld above FP8MI_NORM_MAX_COLS %lld", (long long)cols,
                (long long)kNormMaxCols);
  if (!weight) return FP8MI_OK;
  if (!valid_dtype(dt)) return fail(FP8MI_ERR_ENUM, "weight_dtype %d is not FP8MI_F32/F16/BF16", dt);
  if (reinterpret_cast<uintptr_t>(weight) % dtype_bytes(dt))
    return fail(FP8MI_ERR_ARG, "weight not aligned to its element size");
  return FP8MI_OK;
}

// act: an activation, optionally gated.
static fp8mi_status check_act(int act, int* kind, bool* gated) {
  *gated = act >= 0 && (act & FP8MI_ACT_GATED) != 0;
  *kind = act & ~FP8MI_ACT_GATED;
  if (act < 0 || *kind > FP8MI_ACT_SILU) return fail(FP8MI_ERR_ENUM, "act %d is not an FP8MI_ACT value", act);
  return FP8MI_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static fp8mi_status check_outputs(int mode, int64_t rows, int64_t cols, const uint8_t* out_row, int64_t ld_row,
                                  const uint8_t* out_t, int64_t ld_t, const float* scale_inv_out,
                                  const float* amax_out) {
  const bool any = rows > 0 && cols > 0;
  if (mode != 1) {
    if (any && !out_row) return fail(FP8MI_ERR_NULL, "row-layout output is NULL");
    if (rows > 0 && ld_row < cols) return fail(FP8MI_ERR_SHAPE, "row-layout ld %lld < cols %lld", (long long)ld_row,
                                               (long long)cols);
  }
  if (mode != 0) {
    if (any && !out_t) return fail(FP8MI_ERR_NULL, "transposed output is NULL");
    if (cols > 0 && ld_t < rows) return fail(FP8MI_ERR_SHAPE, "transposed ld %lld < rows %lld", (long long)ld_t,
                                             (long long)rows);
  }
  if ((mode != 1 && !span_ok(rows, ld_row, 1)) || (mode != 0 && !span_ok(cols, ld_t, 1)))
    return fail(FP8MI_ERR_SHAPE, "output extent beyond 2^62 bytes");
  if (reinterpret_cast<uintptr_t>(scale_inv_out) & 3u || reinterpret_cast<uintptr_t>(amax_out) & 3u)
    return fail(FP8MI_ERR_ARG, "fp32 scalars must be 4-byte aligned");
  return FP8MI_OK;
}

static fp8mi_status check_quantize(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, int fmt,
                                   int mode, const uint8_t* out_row, int64_t ld_row, const uint8_t* out_t,
                                   int64_t ld_t, const float* scale, uint32_t* ring, int32_t H,
                                   const float* scale_inv_out, const float* amax_out) {
  fp8mi_status s = check_input(x, dt, rows, cols, ld_x);
  if (s != FP8MI_OK) return s;
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  s = check_scale_ring(scale, ring, H);
  if (s != FP8MI_OK) return s;
  s = check_outputs(mode, rows, cols, out_row, ld_row, out_t, ld_t, scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  if (reinterpret_cast<uintptr_t>(scale) & 3u) return fail(FP8MI_ERR_ARG, "fp32 scalars must be 4-byte aligned");
  return FP8MI_OK;
}

static fp8mi_status quantize_common(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, int fmt,
                                    int mode, uint8_t* out_row, int64_t ld_row, uint8_t* out_t, int64_t ld_t,
                                    const float* scale, uint32_t* ring, int32_t H, float* scale_inv_out,
                                    float* amax_out, void* stream, double* bias_ws = nullptr) {
  fp8mi_status s = check_quantize(x, dt, rows, cols, ld_x, fmt, mode, out_row, ld_row, out_t, ld_t, scale, ring, H,
                                  scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  hipError_t e = launch_quantize(x, dt, rows, cols, ld_x, fmt, mode, out_row, ld_row, out_t, ld_t, scale, ring, H,
                                 scale_inv_out, amax_out, static_cast<hipStream_t>(stream), bias_ws);
  return from_hip(e, "quantize launch");
}

// Bias-gradient arguments shared by fp8_bias_grad and the fused dual
// quantizes, apart from the workspace.
static fp8mi_status check_bias_grad_args(int dt, int64_t rows, int64_t cols, const void* out) {
  if (dt == FP8MI_F32) return fail(FP8MI_ERR_UNSUPPORTED, "the bias gradient takes bf16 or fp16 gradients");
  if (cols > 0 && !out) return fail(FP8MI_ERR_NULL, "bias gradient output is NULL");
  if (reinterpret_cast<uintptr_t>(out) & 1u) return fail(FP8MI_ERR_ARG, "bias gradient output must be 2-byte aligned");
  if ((cols + 511) / 512 > 0x7FFFFFFF || (rows + 127) / 128 > 65535)
    return fail(FP8MI_ERR_UNSUPPORTED, "rows=%lld cols=%lld beyond the launch grid", (long long)rows,
                (long long)cols);
  return FP8MI_OK;
}

static fp8mi_status check_bias_grad(int dt, int64_t rows, int64_t cols, const void* out, const void* workspace,
                                    size_t workspace_bytes) {
  fp8mi_status s = check_bias_grad_args(dt, rows, cols, out);
  if (s != FP8MI_OK) return s;
  const size_t need = (size_t)grad_bias_workspace_bytes(rows, cols);
  if (need > 0 && !workspace) return fail(FP8MI_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
  if (workspace_bytes < need)
    return fail(FP8MI_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 7u) return fail(FP8MI_ERR_ARG, "workspace must be 8-byte aligned");
  return FP8MI_OK;
}

// ---------------------------------------------------------------------------
// Library-owned scratch of fp8_quantize_dual_bias_grad_noalloc: the per-tile
// fp64 column sums that fp8_quantize_dual_bias_grad keeps in the caller's
// workspace.  Every device the library runs on holds its own copy until the
// process ends.  In host code `scratch` names a host-side stand-in, not
// device memory: its device address comes from hipGetSymbolAddress, once
// per device with that device current, and only that address is used.
// ---------------------------------------------------------------------------
static __device__ __align__(256) double scratch[FP8MI_NOALLOC_SCRATCH_BYTES / sizeof(double)];

static fp8mi_status scratch_of_current_device(double** out) {
  static std::mutex mu;
  static std::vector<double*> addr;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return from_hip(e, "hipGetDevice");
  std::lock_guard<std::mutex> lock(mu);
  if ((int)addr.size() <= dev) addr.resize(dev + 1, nullptr);
  if (!addr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return from_hip(e, "hipGetSymbolAddress(scratch)");
    if (!p) return fail(FP8MI_ERR_HIP, "hipGetSymbolAddress(scratch) returned NULL");
    addr[dev] = static_cast<double*>(p);
  }
  *out = addr[dev];
  return FP8MI_OK;
}

}  // namespace fp8mi

using namespace fp8mi;

extern "C" {

fp8mi_status fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, int fmt,
                          int transposed, uint8_t* out, int64_t ld_out, const float* scale, uint32_t* ring,
                          int32_t hist_len, float* scale_inv_out, float* amax_out, void* stream) {
  if (transposed != 0 && transposed != 1) return fail(FP8MI_ERR_ENUM, "transposed must be 0 or 1, got %d", transposed);
  if (transposed)
    return quantize_common(x, x_dtype, rows, cols, ld_x, fmt, 1, nullptr, 0, out, ld_out, scale, ring, hist_len,
                           scale_inv_out, amax_out, stream);
  return quantize_common(x, x_dtype, rows, cols, ld_x, fmt, 0, out, ld_out, nullptr, 0, scale, ring, hist_len,
                         scale_inv_out, amax_out, stream);
}

fp8mi_status fp8_quantize_dynamic(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, int fmt,
                                  int layout, uint8_t* out_row, int64_t ld_row, uint8_t* out_t, int64_t ld_t,
                                  float* scale_inv_out, float* amax_out, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (layout < 0 || layout > 2) return fail(FP8MI_ERR_ENUM, "layout must be 0, 1 or 2, got %d", layout);
  fp8mi_status s = check_input(x, x_dtype, rows, cols, ld_x);
  if (s != FP8MI_OK) return s;
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  s = check_outputs(layout, rows, cols, out_row, ld_row, out_t, ld_t, scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  const size_t need = (size_t)kDynWorkspaceBytes;
  if (!workspace) return fail(FP8MI_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
  if (workspace_bytes < need) return fail(FP8MI_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 3u) return fail(FP8MI_ERR_ARG, "workspace must be 4-byte aligned");
  return from_hip(launch_quantize_dynamic(x, x_dtype, rows, cols, ld_x, fmt, layout, out_row, ld_row, out_t, ld_t,
                                          scale_inv_out, amax_out, static_cast<uint32_t*>(workspace),
                                          static_cast<hipStream_t>(stream)),
                  "dynamic quantize launch");
}

fp8mi_status fp8_quantize_dual(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, int fmt,
                               uint8_t* out_row, int64_t ld_row, uint8_t* out_t, int64_t ld_t, const float* scale,
                               uint32_t* ring, int32_t hist_len, float* scale_inv_out, float* amax_out,
                               void* stream) {
  return quantize_common(x, x_dtype, rows, cols, ld_x, fmt, 2, out_row, ld_row, out_t, ld_t, scale, ring, hist_len,
                         scale_inv_out, amax_out, stream);
}

fp8mi_status fp8_quantize_dual_bias_grad(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                         int fmt, uint8_t* out_row, int64_t ld_row, uint8_t* out_t, int64_t ld_t,
                                         const float* scale, uint32_t* ring, int32_t hist_len, float* scale_inv_out,
                                         float* amax_out, void* bias_grad_out, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  if (!valid_dtype(x_dtype)) return fail(FP8MI_ERR_ENUM, "x_dtype %d is not F32/F16/BF16", x_dtype);
  fp8mi_status s = check_bias_grad(x_dtype, rows, cols, bias_grad_out, workspace, workspace_bytes);
  if (s != FP8MI_OK) return s;
  s = quantize_common(x, x_dtype, rows, cols, ld_x, fmt, 2, out_row, ld_row, out_t, ld_t, scale, ring, hist_len,
                      scale_inv_out, amax_out, stream, static_cast<double*>(workspace));
  if (s != FP8MI_OK || cols == 0) return s;
  return from_hip(launch_grad_bias_finalize(static_cast<const double*>(workspace), rows, cols,
                                            static_cast<uint16_t*>(bias_grad_out), static_cast<hipStream_t>(stream)),
                  "bias grad finalize launch");
}

fp8mi_status fp8_quantize_dual_bias_grad_noalloc(const void* x, int x_dtype, int64_t rows, int64_t cols,
                                                 int64_t ld_x, int fmt, uint8_t* out_row, int64_t ld_row,
                                                 uint8_t* out_t, int64_t ld_t, const float* scale, uint32_t* ring,
                                                 int32_t hist_len, float* scale_inv_out, float* amax_out,
                                                 void* bias_grad_out, void* stream) {
  if (!valid_dtype(x_dtype)) return fail(FP8MI_ERR_ENUM, "x_dtype %d is not F32/F16/BF16", x_dtype);
  fp8mi_status s = check_bias_grad_args(x_dtype, rows, cols, bias_grad_out);
  if (s != FP8MI_OK) return s;
  s = check_quantize(x, x_dtype, rows, cols, ld_x, fmt, 2, out_row, ld_row, out_t, ld_t, scale, ring, hist_len,
                     scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  const size_t need = (size_t)grad_bias_workspace_bytes(rows, cols);
  if (need > (size_t)FP8MI_NOALLOC_SCRATCH_BYTES)
    return fail(FP8MI_ERR_UNSUPPORTED,
                "rows=%lld cols=%lld need %zu bytes of bias-gradient scratch, above the library's %zu; "
                "use fp8_quantize_dual_bias_grad with a caller workspace",
                (long long)rows, (long long)cols, need, (size_t)FP8MI_NOALLOC_SCRATCH_BYTES);
  double* ws = nullptr;
  if (need > 0) {
    s = scratch_of_current_device(&ws);
    if (s != FP8MI_OK) return s;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  s = from_hip(launch_quantize(x, x_dtype, rows, cols, ld_x, fmt, 2, out_row, ld_row, out_t, ld_t, scale, ring,
                               hist_len, scale_inv_out, amax_out, st, ws),
               "quantize launch");
  if (s != FP8MI_OK || cols == 0) return s;
  return from_hip(launch_grad_bias_finalize(ws, rows, cols, static_cast<uint16_t*>(bias_grad_out), st),
                  "bias grad finalize launch");
}

fp8mi_status fp8_amax_fold(uint32_t* ring, int32_t hist_len, const float* amax, int fmt, void* stream) {
  if (!ring) return fail(FP8MI_ERR_NULL, "ring is NULL");
  if (!amax) return fail(FP8MI_ERR_NULL, "amax is NULL");
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  fp8mi_status s = check_scale_ring(nullptr, ring, hist_len);
  if (s != FP8MI_OK) return s;
  return from_hip(launch_amax_fold(ring, hist_len, amax, fmt, static_cast<hipStream_t>(stream)), "fold launch");
}

fp8mi_status fp8_mm_ex(const uint8_t* a, int fmt_a, int64_t lda, int64_t stride_a, const uint8_t* b, int fmt_b,
                       int64_t ldb, int64_t stride_b, int64_t M, int64_t N, int64_t K, int64_t batch, int layout,
                       const float* a_scale_inv, const float* b_scale_inv, const void* bias, int bias_dtype,
                       const float* bias_scale, void* c, int c_dtype, int64_t ldc, int64_t stride_c,
                       const float* c_scale, uint32_t* c_ring, int32_t c_hist_len, float* c_scale_inv_out,
                       float* c_amax_out, void* stream) {
  if (!valid_fmt(fmt_a) || !valid_fmt(fmt_b))
    return fail(FP8MI_ERR_ENUM, "fmt_a %d / fmt_b %d must be FP8MI_E4M3/FP8MI_E5M2", fmt_a, fmt_b);
  if (layout < 0 || layout > 3) return fail(FP8MI_ERR_ENUM, "layout %d is not a combination of FP8MI_A_KM / FP8MI_B_KM", layout);
  const bool fp8_bias = bias_dtype == FP8MI_FP8_E4M3 || bias_dtype == FP8MI_FP8_E5M2;
  if (bias && !valid_dtype(bias_dtype) && !fp8_bias)
    return fail(FP8MI_ERR_ENUM, "bias_dtype %d is not F32/F16/BF16/FP8_E4M3/FP8_E5M2", bias_dtype);
  if (bias && fp8_bias && !bias_scale) return fail(FP8MI_ERR_NULL, "an fp8 bias needs bias_scale");
  if (bias_scale && !(bias && fp8_bias))
    return fail(FP8MI_ERR_ARG, "bias_scale is only for an fp8-stored bias (null scale = raw bias)");
  const bool fp8_out = c_dtype == FP8MI_FP8_E4M3 || c_dtype == FP8MI_FP8_E5M2;
  if (c_dtype != FP8MI_BF16 && !fp8_out) return fail(FP8MI_ERR_ENUM, "c_dtype %d is not BF16/FP8_E4M3/FP8_E5M2", c_dtype);
  if (fp8_out) {
    fp8mi_status s = check_scale_ring(c_scale, c_ring, c_hist_len);
    if (s != FP8MI_OK) return s;
  } else if (c_scale || c_ring || c_scale_inv_out || c_amax_out) {
    return fail(FP8MI_ERR_ARG, "output scale, ring, scale_inv and amax are for an fp8 output only");
  }
  if (M < 0 || N < 0 || K < 0 || batch < 0)
    return fail(FP8MI_ERR_SHAPE, "negative size M=%lld N=%lld K=%lld batch=%lld", (long long)M, (long long)N,
                (long long)K, (long long)batch);
  if ((reinterpret_cast<uintptr_t>(c_scale) | reinterpret_cast<uintptr_t>(c_scale_inv_out) |
       reinterpret_cast<uintptr_t>(c_amax_out) | reinterpret_cast<uintptr_t>(bias_scale)) & 3u)
    return fail(FP8MI_ERR_ARG, "fp32 scalars must be 4-byte aligned");
  MmArgs p;
  p.M = M; p.N = N; p.K = K; p.batch = batch;
  p.out_fmt = fp8_out ? (c_dtype == FP8MI_FP8_E4M3 ? (int)FP8MI_E4M3 : (int)FP8MI_E5M2) : -1;
  p.c_scale = c_scale; p.c_ring = c_ring; p.c_H = c_hist_len;
  p.c_scale_inv_out = c_scale_inv_out; p.c_amax_out = c_amax_out;
  if (M == 0 || N == 0 || batch == 0) {
    // nothing to compute; an fp8 output still completes its scale bookkeeping
    if (!fp8_out) return FP8MI_OK;
    return from_hip(launch_mm(p, fmt_a, fmt_b, static_cast<hipStream_t>(stream)), "mm launch");
  }
  if (!c) return fail(FP8MI_ERR_NULL, "c is NULL");
  if (K > 0 && (!a || !b)) return fail(FP8MI_ERR_NULL, "a or b is NULL");
  if (ldc < N) return fail(FP8MI_ERR_SHAPE, "ldc %lld < N %lld", (long long)ldc, (long long)N);
  const int64_t row_a = (layout & 1) ? M : K, row_b = (layout & 2) ? N : K;  // bytes per stored row
  if (K > 0 && (lda < row_a || ldb < row_b))
    return fail(FP8MI_ERR_SHAPE, "lda %lld / ldb %lld shorter than a stored row (%lld / %lld)", (long long)lda,
                (long long)ldb, (long long)row_a, (long long)row_b);
  if (stride_a < 0 || stride_b < 0 || stride_c < 0) return fail(FP8MI_ERR_STRIDE, "negative batch stride");
  const int64_t elem_c = fp8_out ? 1 : 2;
  const bool reads = K > 0;  // A and B are not read when K = 0
  if ((reads && (!span_ok((layout & 1) ? K : M, lda, 1) || !span_ok((layout & 2) ? K : N, ldb, 1) ||
                 !span_ok(batch, stride_a, 1) || !span_ok(batch, stride_b, 1))) ||
      !span_ok(M, ldc, elem_c) || !span_ok(batch, stride_c, elem_c))
    return fail(FP8MI_ERR_SHAPE, "an operand or output extent is beyond 2^62 bytes");
  if (batch > 1 && stride_c < M * ldc)
    return fail(FP8MI_ERR_STRIDE, "stride_c %lld < M*ldc %lld: batches would overlap", (long long)stride_c,
                (long long)(M * ldc));
  if (!fp8_out && (reinterpret_cast<uintptr_t>(c) & 1u)) return fail(FP8MI_ERR_ARG, "c must be 2-byte aligned");
  if (bias && !fp8_bias && (reinterpret_cast<uintptr_t>(bias) % dtype_bytes(bias_dtype)))
    return fail(FP8MI_ERR_ARG, "bias not aligned to its element size");
  if (K > 0) {
    if ((K % 16) || (lda % 16) || (ldb % 16))
      return fail(FP8MI_ERR_UNSUPPORTED, "K, lda and ldb must be multiples of 16 (K=%lld lda=%lld ldb=%lld)",
                  (long long)K, (long long)lda, (long long)ldb);
    if ((reinterpret_cast<uintptr_t>(a) & 15u) || (reinterpret_cast<uintptr_t>(b) & 15u))
      return fail(FP8MI_ERR_UNSUPPORTED, "a and b must be 16-byte aligned");
    if ((stride_a % 16) || (stride_b % 16))
      return fail(FP8MI_ERR_UNSUPPORTED, "batch strides of a and b must be multiples of 16");
  }
  // the smallest tile is 64 x 64: its count bounds every kernel's grid; below
  // 2^29 per batch, the kernels' tile arithmetic fits 32 bits (no allocation
  // of one GPU comes near: 2^29 such tiles are 4 TB of bf16 output)
  if ((M + 63) / 64 > 65535 || batch > 65535 || (N + 63) / 64 > 0x1FFFFFFF / ((M + 63) / 64))
    return fail(FP8MI_ERR_UNSUPPORTED, "M=%lld N=%lld batch=%lld beyond the launch grid", (long long)M, (long long)N,
                (long long)batch);
  p.a = a; p.b = b; p.lda = lda; p.ldb = ldb; p.stride_a = stride_a; p.stride_b = stride_b;
  p.a_scale_inv = a_scale_inv; p.b_scale_inv = b_scale_inv;
  p.bias = bias; p.bias_dtype = bias ? bias_dtype : -1; p.bias_scale = bias_scale;
  p.c = c; p.ldc = ldc; p.stride_c = stride_c;
  p.layout = layout;
  const int64_t ext_a = (layout & 1) ? p.a_extent_km(0) : p.a_extent_from(0);
  const int64_t ext_b = (layout & 2) ? p.b_extent_km(0) : p.b_extent_from(0);
  if ((fp8_out || layout != 0) && !(ext_a < (1ll << 31) && ext_b < (1ll << 31) && K < (1ll << 30)))
    return fail(FP8MI_ERR_UNSUPPORTED, "an fp8 output or a K-major operand needs operand extents below 2^31 bytes");
  return from_hip(launch_mm(p, fmt_a, fmt_b, static_cast<hipStream_t>(stream)), "mm launch");
}

fp8mi_status fp8_mm(const uint8_t* a, int fmt_a, int64_t lda, int64_t stride_a, const uint8_t* b, int fmt_b,
                    int64_t ldb, int64_t stride_b, int64_t M, int64_t N, int64_t K, int64_t batch,
                    const float* a_scale_inv, const float* b_scale_inv, const void* bias, int bias_dtype, void* c,
                    int64_t ldc, int64_t stride_c, void* stream) {
  if (bias && !valid_dtype(bias_dtype)) return fail(FP8MI_ERR_ENUM, "bias_dtype %d is not F32/F16/BF16", bias_dtype);
  return fp8_mm_ex(a, fmt_a, lda, stride_a, b, fmt_b, ldb, stride_b, M, N, K, batch, 0, a_scale_inv, b_scale_inv, bias,
                   bias_dtype, nullptr, c, FP8MI_BF16, ldc, stride_c, nullptr, nullptr, 0, nullptr, nullptr, stream);
}

size_t fp8_bias_grad_workspace_bytes(int64_t rows, int64_t cols) {
  return (size_t)fp8mi::grad_bias_workspace_bytes(rows, cols);
}

fp8mi_status fp8_bias_grad(const void* dy, int dy_dtype, int64_t rows, int64_t cols, int64_t ld, void* out,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dy_dtype)) return fail(FP8MI_ERR_ENUM, "dy_dtype %d is not F32/F16/BF16", dy_dtype);
  if (dy_dtype == FP8MI_F32) return fail(FP8MI_ERR_UNSUPPORTED, "fp8_bias_grad takes bf16 or fp16 gradients");
  if (rows < 0 || cols < 0) return fail(FP8MI_ERR_SHAPE, "negative shape rows=%lld cols=%lld", (long long)rows,
                                        (long long)cols);
  if (cols == 0) return FP8MI_OK;
  if (!out) return fail(FP8MI_ERR_NULL, "out is NULL");
  if (rows > 0 && !dy) return fail(FP8MI_ERR_NULL, "dy is NULL");
  if (rows > 0 && ld < cols) return fail(FP8MI_ERR_SHAPE, "ld %lld < cols %lld", (long long)ld, (long long)cols);
  if (!span_ok(rows, ld, 2)) return fail(FP8MI_ERR_SHAPE, "rows %lld x ld %lld beyond 2^62 bytes", (long long)rows,
                                         (long long)ld);
  if (reinterpret_cast<uintptr_t>(dy) & 1u) return fail(FP8MI_ERR_ARG, "dy must be 2-byte aligned");
  fp8mi_status s = check_bias_grad(dy_dtype, rows, cols, out, workspace, workspace_bytes);
  if (s != FP8MI_OK) return s;
  return from_hip(launch_grad_bias(dy, dy_dtype, rows, cols, ld, static_cast<uint16_t*>(out), workspace,
                                   static_cast<hipStream_t>(stream)),
                  "bias grad launch");
}

fp8mi_status fp8_rmsnorm(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                         int64_t ld_res, const void* weight, int weight_dtype, const float* eps, int fmt, uint8_t* out,
                         int64_t ld_out, int scaling, const float* scale, uint32_t* ring, int32_t hist_len,
                         float* scale_inv_out, float* amax_out, void* sum_out, int64_t ld_sum, float* rstd_out,
                         void* stream) {
  fp8mi_status s = check_input(x, x_dtype, rows, cols, ld_x);
  if (s != FP8MI_OK) return s;
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  s = check_norm_weight(weight, weight_dtype, cols);
  if (s != FP8MI_OK) return s;
  if (!eps) return fail(FP8MI_ERR_NULL, "eps is NULL");
  if (!(*eps >= 0.0f)) return fail(FP8MI_ERR_ARG, "eps %g is not a number >= 0", (double)*eps);
  if (scaling == FP8MI_SCALE_TENSOR) {
    s = check_scale_ring(scale, ring, hist_len);
    if (s != FP8MI_OK) return s;
    if (!aligned4(scale)) return fail(FP8MI_ERR_ARG, "fp32 scalars must be 4-byte aligned");
  } else if (scaling == FP8MI_SCALE_ROW) {
    if (scale || ring) return fail(FP8MI_ERR_ARG, "row scaling measures its scales: give neither scale nor ring");
    if (rows > 0 && !scale_inv_out) return fail(FP8MI_ERR_NULL, "row scaling needs scale_inv_out [rows]");
  } else {
    return fail(FP8MI_ERR_ENUM, "scaling %d is not FP8MI_SCALE_TENSOR/FP8MI_SCALE_ROW", scaling);
  }
  s = check_outputs(0, rows, cols, out, ld_out, nullptr, 0, scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  s = check_matrix("residual", residual, false, x_dtype, rows, cols, ld_res);
  if (s != FP8MI_OK) return s;
  s = check_matrix("sum_out", sum_out, false, x_dtype, rows, cols, ld_sum);
  if (s != FP8MI_OK) return s;
  if (!aligned4(rstd_out)) return fail(FP8MI_ERR_ARG, "rstd_out must be 4-byte aligned");
  NormArgs p;
  p.x = x; p.res = residual; p.weight = weight; p.weight_dt = weight_dtype;
  p.rows = rows; p.cols = cols; p.ld_x = ld_x; p.ld_res = ld_res;
  p.eps = *eps; p.n_cols = cols > 0 ? (float)cols : 1.0f;
  p.out = out; p.ld_out = ld_out; p.fmt = fmt;
  p.row_scaled = scaling == FP8MI_SCALE_ROW; p.scale = scale; p.ring = ring; p.H = hist_len;
  p.scale_inv_out = scale_inv_out; p.amax_out = amax_out;
  p.sum_out = sum_out; p.ld_sum = ld_sum; p.rstd_out = rstd_out;
  return from_hip(launch_rmsnorm(p, x_dtype, static_cast<hipStream_t>(stream)), "rmsnorm launch");
}

fp8mi_status fp8_mm_act(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int64_t M, int64_t N, int64_t K,
                        const float* a_scale_inv, const float* b_scale_inv, int scale_rows, const void* bias,
                        int bias_dtype, int act, const void* residual, int residual_dtype, int64_t ld_res, void* z_out,
                        int64_t ld_z, void* c, int c_dtype, int64_t ldc, const float* c_scale, uint32_t* c_ring,
                        int32_t c_hist_len, float* c_scale_inv_out, float* c_amax_out, void* stream) {
  int kind;
  bool gated;
  fp8mi_status s = check_act(act, &kind, &gated);
  if (s != FP8MI_OK) return s;
  if (scale_rows < 0 || scale_rows > 3)
    return fail(FP8MI_ERR_ENUM, "scale_rows %d is not a combination of FP8MI_A_ROW_SCALES / FP8MI_B_ROW_SCALES", scale_rows);
  if (((scale_rows & FP8MI_A_ROW_SCALES) && !a_scale_inv) || ((scale_rows & FP8MI_B_ROW_SCALES) && !b_scale_inv))
    return fail(FP8MI_ERR_NULL, "row scales are announced but their array is NULL");
  if (bias && !valid_dtype(bias_dtype)) return fail(FP8MI_ERR_ENUM, "bias_dtype %d is not F32/F16/BF16", bias_dtype);
  if (residual && !valid_dtype(residual_dtype))
    return fail(FP8MI_ERR_ENUM, "residual_dtype %d is not F32/F16/BF16", residual_dtype);
  const bool fp8_out = c_dtype == FP8MI_FP8_E4M3;
  if (c_dtype == FP8MI_FP8_E5M2) return fail(FP8MI_ERR_UNSUPPORTED, "fp8_mm_act's fp8 output is E4M3");
  if (c_dtype != FP8MI_BF16 && !fp8_out) return fail(FP8MI_ERR_ENUM, "c_dtype %d is not BF16/FP8_E4M3", c_dtype);
  if (fp8_out) {
    s = check_scale_ring(c_scale, c_ring, c_hist_len);
    if (s != FP8MI_OK) return s;
  } else if (c_scale || c_ring || c_scale_inv_out || c_amax_out) {
    return fail(FP8MI_ERR_ARG, "output scale, ring, scale_inv and amax are for an fp8 output only");
  }
  if (M < 0 || N < 0 || K < 0)
    return fail(FP8MI_ERR_SHAPE, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (gated && (N & 1)) return fail(FP8MI_ERR_SHAPE, "a gated product needs an even N, got %lld", (long long)N);
  const int64_t No = gated ? N / 2 : N;
  if (!aligned4(a_scale_inv) || !aligned4(b_scale_inv) || !aligned4(c_scale) || !aligned4(c_scale_inv_out) ||
      !aligned4(c_amax_out))
    return fail(FP8MI_ERR_ARG, "fp32 scales must be 4-byte aligned");
  if (M > 0 && N > 0) {
    if (!c) return fail(FP8MI_ERR_NULL, "c is NULL");
    if (K > 0 && (!a || !b)) return fail(FP8MI_ERR_NULL, "a or b is NULL");
    if (ldc < No) return fail(FP8MI_ERR_SHAPE, "ldc %lld < outputs %lld", (long long)ldc, (long long)No);
    if (K > 0 && (lda < K || ldb < K))
      return fail(FP8MI_ERR_SHAPE, "lda %lld / ldb %lld < K %lld", (long long)lda, (long long)ldb, (long long)K);
    if ((K > 0 && (!span_ok(M, lda, 1) || !span_ok(N, ldb, 1))) || !span_ok(M, ldc, fp8_out ? 1 : 2))
      return fail(FP8MI_ERR_SHAPE, "an operand or output extent is beyond 2^62 bytes");
    s = check_matrix("z_out", z_out, false, FP8MI_BF16, M, N, ld_z);
    if (s != FP8MI_OK) return s;
    if (residual) {
      s = check_matrix("residual", residual, false, residual_dtype, M, No, ld_res);
      if (s != FP8MI_OK) return s;
    }
    if (!fp8_out && (reinterpret_cast<uintptr_t>(c) & 1u)) return fail(FP8MI_ERR_ARG, "c must be 2-byte aligned");
    if (bias && reinterpret_cast<uintptr_t>(bias) % dtype_bytes(bias_dtype))
      return fail(FP8MI_ERR_ARG, "bias not aligned to its element size");
    if (K > 0) {
      if ((K % 16) || (lda % 16) || (ldb % 16))
        return fail(FP8MI_ERR_UNSUPPORTED, "K, lda and ldb must be multiples of 16 (K=%lld lda=%lld ldb=%lld)",
                    (long long)K, (long long)lda, (long long)ldb);
      if ((reinterpret_cast<uintptr_t>(a) & 15u) || (reinterpret_cast<uintptr_t>(b) & 15u))
        return fail(FP8MI_ERR_UNSUPPORTED, "a and b must be 16-byte aligned");
    }
    if ((M + 63) / 64 > 65535 || (N + 31) / 32 > 0x1FFFFFFF / ((M + 63) / 64))
      return fail(FP8MI_ERR_UNSUPPORTED, "M=%lld N=%lld beyond the launch grid", (long long)M, (long long)N);
  }
  MmActArgs p;
  p.a = a; p.b = b; p.lda = lda; p.ldb = ldb; p.M = M; p.N = N; p.K = K; p.batch = 1;
  p.a_scale_inv = a_scale_inv; p.b_scale_inv = b_scale_inv;
  p.a_rows = (scale_rows & FP8MI_A_ROW_SCALES) != 0; p.b_rows = (scale_rows & FP8MI_B_ROW_SCALES) != 0;
  p.bias = bias; p.bias_dtype = bias ? bias_dtype : -1;
  p.act = kind; p.res = residual; p.res_dt = residual_dtype; p.ld_res = ld_res;
  p.z = static_cast<uint16_t*>(z_out); p.ld_z = ld_z;
  p.c = c; p.ldc = ldc; p.out_fmt = fp8_out ? (int)FP8MI_E4M3 : -1;
  p.c_scale = c_scale; p.c_ring = c_ring; p.c_H = c_hist_len;
  p.c_scale_inv_out = c_scale_inv_out; p.c_amax_out = c_amax_out;
  if (M > 0 && N > 0 &&
      !(p.a_extent_from(0) < (1ll << 31) && p.b_extent_from(0) < (1ll << 31) && K < (1ll << 30)))
    return fail(FP8MI_ERR_UNSUPPORTED, "fp8_mm_act needs operand extents below 2^31 bytes");
  return from_hip(launch_mm_act(p, gated, static_cast<hipStream_t>(stream)), "mm_act launch");
}

fp8mi_status fp8_act_grad(const void* dy, int dy_dtype, int64_t rows, int64_t cols, int64_t ld_dy, const void* z,
                          int64_t ld_z, int act, int fmt, uint8_t* out_row, int64_t ld_row, uint8_t* out_t,
                          int64_t ld_t, const float* scale, uint32_t* ring, int32_t hist_len, float* scale_inv_out,
                          float* amax_out, void* bias_grad_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int kind;
  bool gated;
  fp8mi_status s = check_act(act, &kind, &gated);
  if (s != FP8MI_OK) return s;
  if (kind == FP8MI_ACT_NONE && !gated)
    return fail(FP8MI_ERR_ARG, "without an activation dz is dy: use fp8_quantize_dual");
  if (gated && (cols & 1)) return fail(FP8MI_ERR_SHAPE, "a gated gradient needs an even cols, got %lld", (long long)cols);
  s = check_input(dy, dy_dtype, rows, gated ? cols / 2 : cols, ld_dy);
  if (s != FP8MI_OK) return s;
  if (dy_dtype == FP8MI_F32) return fail(FP8MI_ERR_UNSUPPORTED, "fp8_act_grad takes bf16 or fp16 gradients");
  s = check_matrix("z", z, true, FP8MI_BF16, rows, cols, ld_z);
  if (s != FP8MI_OK) return s;
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  s = check_scale_ring(scale, ring, hist_len);
  if (s != FP8MI_OK) return s;
  if (!aligned4(scale)) return fail(FP8MI_ERR_ARG, "fp32 scalars must be 4-byte aligned");
  s = check_outputs(2, rows, cols, out_row, ld_row, out_t, ld_t, scale_inv_out, amax_out);
  if (s != FP8MI_OK) return s;
  if ((rows + 127) / 128 > 0 && (cols + 63) / 64 > 0x7FFFFFFF / ((rows + 127) / 128))
    return fail(FP8MI_ERR_UNSUPPORTED, "rows=%lld cols=%lld beyond the launch grid", (long long)rows, (long long)cols);
  if (bias_grad_out) {
    s = check_bias_grad(dy_dtype, rows, cols, bias_grad_out, workspace, workspace_bytes);
    if (s != FP8MI_OK) return s;
  }
  ActGradArgs p;
  p.dy = dy; p.z = static_cast<const uint16_t*>(z); p.rows = rows; p.cols = cols; p.ld_dy = ld_dy; p.ld_z = ld_z;
  p.out_row = out_row; p.ld_row = ld_row; p.out_t = out_t; p.ld_t = ld_t;
  p.scale = scale; p.ring = ring; p.H = hist_len; p.scale_inv_out = scale_inv_out; p.amax_out = amax_out;
  p.bias_ws = bias_grad_out ? static_cast<double*>(workspace) : nullptr;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  s = from_hip(launch_act_grad(p, dy_dtype, fmt, kind, gated, st), "activation gradient launch");
  if (s != FP8MI_OK || !bias_grad_out || cols == 0) return s;
  return from_hip(launch_grad_bias_finalize(p.bias_ws, rows, cols, static_cast<uint16_t*>(bias_grad_out), st),
                  "bias grad finalize launch");
}

size_t fp8_rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  return (size_t)fp8mi::rmsnorm_grad_workspace_bytes(rows, cols);
}

fp8mi_status fp8_rmsnorm_grad(const void* dy, int dtype, int64_t rows, int64_t cols, int64_t ld_dy, const void* h,
                              int64_t ld_h, const void* weight, int weight_dtype, const float* rstd, const void* dsum,
                              int64_t ld_dsum, void* dx, int64_t ld_dx, float* dweight, void* workspace,
                              size_t workspace_bytes, void* stream) {
  fp8mi_status s = check_input(dy, dtype, rows, cols, ld_dy);
  if (s != FP8MI_OK) return s;
  s = check_norm_weight(weight, weight_dtype, cols);
  if (s != FP8MI_OK) return s;
  s = check_matrix("h", h, true, dtype, rows, cols, ld_h);
  if (s != FP8MI_OK) return s;
  s = check_matrix("dsum", dsum, false, dtype, rows, cols, ld_dsum);
  if (s != FP8MI_OK) return s;
  s = check_matrix("dx", dx, true, dtype, rows, cols, ld_dx);
  if (s != FP8MI_OK) return s;
  if (rows > 0 && cols > 0 && !rstd) return fail(FP8MI_ERR_NULL, "rstd is NULL");
  if (!aligned4(rstd) || !aligned4(dweight)) return fail(FP8MI_ERR_ARG, "rstd and dweight must be 4-byte aligned");
  if (dweight) {
    const size_t need = (size_t)rmsnorm_grad_workspace_bytes(rows, cols);
    if (need > 0 && !workspace) return fail(FP8MI_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
    if (workspace_bytes < need)
      return fail(FP8MI_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
    if (!aligned4(workspace)) return fail(FP8MI_ERR_ARG, "workspace must be 4-byte aligned");
  }
  NormGradArgs p;
  p.dy = dy; p.h = h; p.weight = weight; p.weight_dt = weight_dtype; p.rstd = rstd; p.dsum = dsum; p.dx = dx;
  p.rows = rows; p.cols = cols; p.ld_dy = ld_dy; p.ld_h = ld_h; p.ld_dsum = ld_dsum; p.ld_dx = ld_dx;
  p.n_cols = cols > 0 ? (float)cols : 1.0f;
  return from_hip(launch_rmsnorm_grad(p, dtype, dweight, workspace, static_cast<hipStream_t>(stream)),
                  "rmsnorm gradient launch");
}

// Sizes that the cross entropy's kernels, 32-bit offsets and grids (below 2^32 threads)
// cover.
static fp8mi_status check_xent_size(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1 || K < 1)
    return fail(FP8MI_ERR_SHAPE, "M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (K % 16 || K > 65536 || M > (1 << 20) || M >= (INT64_C(1) << 30) / (K + 64) || N > (1 << 28))
    return fail(FP8MI_ERR_UNSUPPORTED, "M=%lld N=%lld K=%lld: K is a multiple of 16 up to 65536, M at most 2^20, M (K + 64) "
                "below 2^30, N at most 2^28", (long long)M, (long long)N, (long long)K);
  return FP8MI_OK;
}

static fp8mi_status check_xent(const XentCall& c, int target_bits, const void* workspace, size_t workspace_bytes,
                               size_t need) {
  const fp8mi_status s = check_xent_size(c.M, c.N, c.K);
  if (s != FP8MI_OK) return s;
  if (target_bits != 32 && target_bits != 64) return fail(FP8MI_ERR_ENUM, "target_bits %d is not 32/64", target_bits);
  if (!aligned4(c.a_scale_inv) || !aligned4(c.b_scale_inv)) return fail(FP8MI_ERR_ARG, "fp32 scales must be 4-byte aligned");
  if (c.M == 0) return FP8MI_OK;
  if (!c.a || !c.b || !c.targets) return fail(FP8MI_ERR_NULL, "a, b or targets is NULL");
  if (c.lda < c.K || c.ldb < c.K)
    return fail(FP8MI_ERR_SHAPE, "lda %lld / ldb %lld < K %lld", (long long)c.lda, (long long)c.ldb, (long long)c.K);
  if (c.lda > (1 << 22) || c.ldb > (1 << 22))
    return fail(FP8MI_ERR_UNSUPPORTED, "lda %lld / ldb %lld above 2^22", (long long)c.lda, (long long)c.ldb);
  if ((c.lda % 16) || (c.ldb % 16) || (reinterpret_cast<uintptr_t>(c.a) & 15u) || (reinterpret_cast<uintptr_t>(c.b) & 15u))
    return fail(FP8MI_ERR_UNSUPPORTED, "a and b must be 16-byte aligned, lda and ldb multiples of 16");
  if (reinterpret_cast<uintptr_t>(c.targets) % (target_bits / 8)) return fail(FP8MI_ERR_ARG, "targets not aligned to their size");
  if (!workspace) return fail(FP8MI_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
  if (workspace_bytes < need) return fail(FP8MI_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return fail(FP8MI_ERR_ARG, "workspace must be 16-byte aligned");
  return FP8MI_OK;
}

size_t fp8_cross_entropy_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M > 0 && check_xent_size(M, N, K) == FP8MI_OK ? (size_t)xent_workspace_bytes(M, N, K) : 0;
}

size_t fp8_cross_entropy_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M > 0 && check_xent_size(M, N, K) == FP8MI_OK ? (size_t)xent_grad_workspace_bytes(M, N, K) : 0;
}

fp8mi_status fp8_cross_entropy(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int64_t M, int64_t N,
                               int64_t K, const float* a_scale_inv, const float* b_scale_inv, int scale_rows,
                               const void* targets, int target_bits, float* loss, float* lse, float* mean_out,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (scale_rows < 0 || scale_rows > 3)
    return fail(FP8MI_ERR_ENUM, "scale_rows %d is not a combination of FP8MI_A_ROW_SCALES / FP8MI_B_ROW_SCALES", scale_rows);
  XentCall c;
  c.a = a; c.b = b; c.lda = lda; c.ldb = ldb; c.M = M; c.N = N; c.K = K;
  c.a_scale_inv = a_scale_inv; c.b_scale_inv = b_scale_inv;
  c.a_rows = (scale_rows & FP8MI_A_ROW_SCALES) != 0; c.b_rows = (scale_rows & FP8MI_B_ROW_SCALES) != 0;
  c.targets = targets; c.target_bits = target_bits; c.ws = static_cast<uint8_t*>(workspace);
  c.loss = loss; c.lse = lse; c.mean = mean_out;
  if ((c.a_rows && !a_scale_inv) || (c.b_rows && !b_scale_inv))
    return fail(FP8MI_ERR_NULL, "row scales are announced but their array is NULL");
  const fp8mi_status s = check_xent(c, target_bits, workspace, workspace_bytes, fp8_cross_entropy_workspace_bytes(M, N, K));
  if (s != FP8MI_OK) return s;
  if (M > 0 && (!loss || !lse)) return fail(FP8MI_ERR_NULL, "loss or lse is NULL");
  if (!aligned4(loss) || !aligned4(lse) || !aligned4(mean_out))
    return fail(FP8MI_ERR_ARG, "loss, lse and mean_out must be 4-byte aligned");
  return from_hip(launch_xent_forward(c, static_cast<hipStream_t>(stream)), "cross entropy launch");
}

fp8mi_status fp8_cross_entropy_grad(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int64_t M, int64_t N,
                                    int64_t K, const float* a_scale_inv, const float* b_scale_inv, const void* targets,
                                    int target_bits, const float* lse, const float* dloss, int dloss_rows, void* da,
                                    int64_t ld_da, void* db, int64_t ld_db, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (dloss_rows != 0 && dloss_rows != 1) return fail(FP8MI_ERR_ENUM, "dloss_rows %d is not 0/1", dloss_rows);
  XentCall c;
  c.a = a; c.b = b; c.lda = lda; c.ldb = ldb; c.M = M; c.N = N; c.K = K;
  c.a_scale_inv = a_scale_inv; c.b_scale_inv = b_scale_inv;
  c.targets = targets; c.target_bits = target_bits; c.ws = static_cast<uint8_t*>(workspace);
  c.lse = const_cast<float*>(lse); c.dloss = dloss; c.dloss_rows = dloss_rows;
  c.da = static_cast<uint16_t*>(da); c.db = static_cast<uint16_t*>(db); c.ld_da = ld_da; c.ld_db = ld_db;
  fp8mi_status s = check_xent(c, target_bits, workspace, workspace_bytes, fp8_cross_entropy_grad_workspace_bytes(M, N, K));
  if (s != FP8MI_OK) return s;
  if (M > 0 && (!lse || !dloss)) return fail(FP8MI_ERR_NULL, "lse or dloss is NULL");
  if (!aligned4(lse) || !aligned4(dloss)) return fail(FP8MI_ERR_ARG, "lse and dloss must be 4-byte aligned");
  s = check_matrix("da", da, false, FP8MI_BF16, M, K, ld_da);
  if (s != FP8MI_OK) return s;
  s = check_matrix("db", db, false, FP8MI_BF16, N, K, ld_db);
  if (s != FP8MI_OK) return s;
  if (!da && !db) return FP8MI_OK;
  return from_hip(launch_xent_backward(c, static_cast<hipStream_t>(stream)), "cross entropy gradient launch");
}

// What grids of 2^31 threads cover: 1024 elements of a tensor, 32768 of all gradients, to
// a workgroup of 256.
constexpr int64_t kAdamWElements = INT64_C(1) << 33, kNormElements = INT64_C(1) << 38;

// One tensor of a list: n elements of dtype at p, at most `most`.
static fp8mi_status check_elements(const char* name, int i, const void* p, int64_t n, int dt, int64_t most) {
  if (!valid_dtype(dt)) return fail(FP8MI_ERR_ENUM, "tensor %d: %s dtype %d is not F32/F16/BF16", i, name, dt);
  if (n < 0 || n > most) return fail(FP8MI_ERR_SHAPE, "tensor %d: %lld elements", i, (long long)n);
  if (n > 0 && !p) return fail(FP8MI_ERR_NULL, "tensor %d: %s is NULL", i, name);
  if (reinterpret_cast<uintptr_t>(p) % dtype_bytes(dt))
    return fail(FP8MI_ERR_ARG, "tensor %d: %s not aligned to its element size", i, name);
  return FP8MI_OK;
}

fp8mi_status fp8_adamw_step(const fp8mi_adamw_tensor* tensors, int32_t count, const fp8mi_adamw* hyper, void* stream) {
  if (!hyper) return fail(FP8MI_ERR_NULL, "hyper is NULL");
  if (count < 0) return fail(FP8MI_ERR_SHAPE, "count %d", count);
  if (count > 0 && !tensors) return fail(FP8MI_ERR_NULL, "tensors is NULL");
  const fp8mi_adamw& h = *hyper;
  if (!(h.beta1 >= 0.0 && h.beta1 < 1.0 && h.beta2 >= 0.0 && h.beta2 < 1.0))
    return fail(FP8MI_ERR_ARG, "betas %g, %g outside [0, 1)", h.beta1, h.beta2);
  if (!(h.eps >= 0.0) || !(h.lr >= 0.0)) return fail(FP8MI_ERR_ARG, "eps %g or lr %g is not a number >= 0", h.eps, h.lr);
  if (h.step_device ? h.step != 0 : (h.step < 1 || h.step > INT64_C(0x7FFFFFFF)))
    return fail(FP8MI_ERR_ARG, "step %lld: a number from 1 on, or 0 with step_device", (long long)h.step);
  if (h.lr_device && !h.step_device) return fail(FP8MI_ERR_ARG, "lr_device needs step_device");
  if (!aligned4(h.step_device) || !aligned4(h.lr_device) || !aligned4(h.grad_scale))
    return fail(FP8MI_ERR_ARG, "device words must be 4-byte aligned");
  for (int i = 0; i < count; ++i) {
    const fp8mi_adamw_tensor& t = tensors[i];
    fp8mi_status s = check_elements("param", i, t.param, t.n, t.param_dtype, kAdamWElements);
    if (s == FP8MI_OK) s = check_elements("grad", i, t.grad, t.n, t.grad_dtype, kAdamWElements);
    if (s != FP8MI_OK) return s;
    if (t.state_bits != 32 && t.state_bits != 8)
      return fail(FP8MI_ERR_ENUM, "tensor %d: state_bits %d is not 32/8", i, t.state_bits);
    const bool bytes = t.state_bits == 8;
    if (t.n > 0 && (!t.exp_avg || !t.exp_avg_sq || (bytes && (!t.exp_avg_scale || !t.exp_avg_sq_scale))))
      return fail(FP8MI_ERR_NULL, "tensor %d: a state or its scales are NULL", i);
    if (!bytes && (t.exp_avg_scale || t.exp_avg_sq_scale))
      return fail(FP8MI_ERR_ARG, "tensor %d: scales belong to 8-bit states", i);
    if (t.master && t.param_dtype == FP8MI_F32)
      return fail(FP8MI_ERR_ARG, "tensor %d: an fp32 param is its own master", i);
    if (!aligned4(t.master) || !aligned4(t.exp_avg_scale) || !aligned4(t.exp_avg_sq_scale) ||
        (!bytes && (!aligned4(t.exp_avg) || !aligned4(t.exp_avg_sq))))
      return fail(FP8MI_ERR_ARG, "tensor %d: masters, fp32 states and scales must be 4-byte aligned", i);
    if (!(t.weight_decay >= 0.0f)) return fail(FP8MI_ERR_ARG, "tensor %d: weight_decay %g", i, (double)t.weight_decay);
  }
  AdamWHyper a;
  a.lr = (float)h.lr; a.beta1 = (float)h.beta1; a.beta2 = (float)h.beta2;
  a.one_beta1 = (float)(1.0 - h.beta1); a.one_beta2 = (float)(1.0 - h.beta2); a.eps = (float)h.eps;
  a.t = (uint32_t)h.step; a.seed = h.seed;
  a.step_size = a.root_scale = 0.0f;
  if (!h.step_device) {
    a.step_size = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
    a.root_scale = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
  }
  a.grad_scale = h.grad_scale; a.step_words = h.step_device; a.lr_word = h.lr_device;
  return from_hip(launch_adamw(tensors, count, a, h.beta1, h.beta2, static_cast<hipStream_t>(stream)), "adamw launch");
}

size_t fp8_grad_norm_workspace_bytes(const fp8mi_norm_tensor* tensors, int32_t count) {
  if (!tensors || count <= 0) return 0;
  for (int i = 0; i < count; ++i)
    if (tensors[i].n < 0 || tensors[i].n > kNormElements) return 0;
  return (size_t)grad_norm_workspace_bytes(tensors, count);
}

fp8mi_status fp8_grad_norm(const fp8mi_norm_tensor* tensors, int32_t count, const float* max_norm, float* norm_out,
                           float* clip_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (count < 0) return fail(FP8MI_ERR_SHAPE, "count %d", count);
  if (count > 0 && !tensors) return fail(FP8MI_ERR_NULL, "tensors is NULL");
  if (max_norm && !(*max_norm >= 0.0f)) return fail(FP8MI_ERR_ARG, "max_norm %g is not a number >= 0", (double)*max_norm);
  if (!aligned4(norm_out) || !aligned4(clip_out)) return fail(FP8MI_ERR_ARG, "fp32 outputs must be 4-byte aligned");
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const fp8mi_status s = check_elements("grad", i, tensors[i].grad, tensors[i].n, tensors[i].dtype, kNormElements);
    if (s != FP8MI_OK) return s;
    total += tensors[i].n;
    if (total > kNormElements) return fail(FP8MI_ERR_SHAPE, "more than 2^38 elements");
  }
  const size_t need = fp8_grad_norm_workspace_bytes(tensors, count);
  if (need > 0 && !workspace) return fail(FP8MI_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
  if (workspace_bytes < need)
    return fail(FP8MI_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 7u) return fail(FP8MI_ERR_ARG, "workspace must be 8-byte aligned");
  return from_hip(launch_grad_norm(tensors, count, max_norm ? *max_norm : -1.0f, norm_out, clip_out,
                                   static_cast<double*>(workspace), static_cast<hipStream_t>(stream)),
                  "gradient norm launch");
}

fp8mi_status fp8_ring_seed(uint32_t* ring, int32_t hist_len, const float* amax, int fmt, void* stream) {
  if (!ring) return fail(FP8MI_ERR_NULL, "ring is NULL");
  if (!amax) return fail(FP8MI_ERR_NULL, "amax is NULL");
  if (!valid_fmt(fmt)) return fail(FP8MI_ERR_ENUM, "fmt %d is not FP8MI_E4M3/FP8MI_E5M2", fmt);
  fp8mi_status s = check_scale_ring(nullptr, ring, hist_len);
  if (s != FP8MI_OK) return s;
  return from_hip(launch_ring_seed(ring, hist_len, amax, fmt, static_cast<hipStream_t>(stream)), "seed launch");
}

fp8mi_status fp8mi_stream_reference(const void* src, int64_t src_bytes, void* dst, int64_t dst_bytes,
                                    void* stream) {
  if (src_bytes < 0 || src_bytes % 16) return fail(FP8MI_ERR_ARG, "src_bytes %lld is not a multiple of 16",
                                                   (long long)src_bytes);
  if (dst_bytes != src_bytes && 2 * dst_bytes != src_bytes)
    return fail(FP8MI_ERR_ARG, "dst_bytes %lld must equal src_bytes %lld or its half", (long long)dst_bytes,
                (long long)src_bytes);
  if (src_bytes == 0) return FP8MI_OK;
  if (!src || !dst) return fail(FP8MI_ERR_NULL, "src or dst is NULL");
  if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u)
    return fail(FP8MI_ERR_ARG, "src and dst must be 16-byte aligned");
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), d0 = reinterpret_cast<uintptr_t>(dst);
  if (s0 < d0 + (uintptr_t)dst_bytes && d0 < s0 + (uintptr_t)src_bytes)
    return fail(FP8MI_ERR_ARG, "src and dst overlap");
  return from_hip(launch_stream(src, src_bytes, dst, dst_bytes, static_cast<hipStream_t>(stream)),
                  "stream reference launch");
}

const char* fp8mi_status_string(int s) {
  switch (s) {
    case FP8MI_OK: return "ok";
    case FP8MI_ERR_NULL: return "required pointer is NULL";
    case FP8MI_ERR_ENUM: return "enum value out of range";
    case FP8MI_ERR_SHAPE: return "invalid shape or leading dimension";
    case FP8MI_ERR_STRIDE: return "invalid batch stride";
    case FP8MI_ERR_UNSUPPORTED: return "unsupported layout or alignment";
    case FP8MI_ERR_HIP: return "HIP runtime error";
    case FP8MI_ERR_ARG: return "inconsistent arguments";
    default: return "unknown status";
  }
}

const char* fp8mi_last_error(void) { return g_err; }

const char* fp8mi_version(void) { return "fp8mi 0.1 gfx950"; }

}  // extern "C"
