// Host side of the 8-bit entry points (include/hyb_f8.h): argument checks,
// then the launch.
#include "hyb_f8_internal.h"

namespace {

using hyb::fail;
using hyb::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_type(int32_t dt) { return dt == HYB_F16 || dt == HYB_BF16 || dt == HYB_F32; }

int elem_size(int32_t dt) { return dt == HYB_F32 ? 4 : 2; }

hyb_status check_shape(int64_t rows, int64_t k) {
  if (rows < 0 || rows > hyb::kF8MaxRows)
    return fail(HYB_ERR_SHAPE, "rows = %lld outside [0, %lld]", (long long)rows, (long long)hyb::kF8MaxRows);
  if (k < 0 || k > hyb::kF8MaxK)
    return fail(HYB_ERR_SHAPE, "k = %lld outside [0, %lld]", (long long)k, (long long)hyb::kF8MaxK);
  return HYB_OK;
}

hyb_status check_f8(const hyb_f8* p, const char* name) {
  if (!p || !p->codes || !p->scales) return fail(HYB_ERR_INVALID_ARG, "%s, its codes or its scales are NULL", name);
  if (!aligned(p->codes, 16) || !aligned(p->scales, 16))
    return fail(HYB_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", name);
  return HYB_OK;
}

hyb_status check_plain(const void* a, int32_t dtype, int64_t k, int64_t ld, const char* name) {
  if (!a || !aligned(a, elem_size(dtype)))
    return fail(HYB_ERR_INVALID_ARG, "%s is NULL or not aligned to its element size", name);
  if (ld < k) return fail(HYB_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)ld, (long long)k);
  if (ld > (int64_t(1) << 31))
    return fail(HYB_ERR_UNSUPPORTED, "%s row stride %lld is above 2^31", name, (long long)ld);
  return HYB_OK;
}

// Checks of a product; the workspace may be absent.
hyb_status check_gemm(const hyb_f8* w, int64_t n, int64_t k, const hyb_f8* x, int32_t m, const void* y, int32_t y_dtype,
                      int64_t ldy, const void* workspace, size_t workspace_bytes) {
  if (!known_type(y_dtype)) return fail(HYB_ERR_DTYPE, "y_dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", y_dtype);
  hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (m < 0) return fail(HYB_ERR_SHAPE, "m = %d is negative", m);
  if (workspace_bytes > 0 && (!workspace || !aligned(workspace, 16)))
    return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned with workspace_bytes = %zu",
                workspace_bytes);
  if (m == 0 || n == 0) return HYB_OK;
  if ((st = check_plain(y, y_dtype, n, ldy, "y")) != HYB_OK) return st;
  if (k > 0) {
    if ((st = check_f8(w, "w")) != HYB_OK) return st;
    if ((st = check_f8(x, "x")) != HYB_OK) return st;
  }
  if (m > hyb::kF8MaxRows || ((n + 15) / 16) * ((int64_t(m) + 15) / 16) >= hyb::kF8MaxPanelPairs)
    return fail(HYB_ERR_UNSUPPORTED, "n x m = %lld x %d is too large for one launch", (long long)n, m);
  const size_t need = k > 0 ? hyb::f8_workspace_bytes(n, k, m, hyb::device_cus()) : 0;
  if (workspace_bytes > 0 && workspace_bytes < need)
    return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this product needs %zu (or 0: unsplit)", workspace_bytes,
                need);
  return HYB_OK;
}

// hyb_f8_linear's quantised activations at the start of its workspace: their
// bytes, and their addresses.
size_t linear_scratch(int64_t k, int64_t m, hyb_f8* x, char* base = nullptr) {
  const int64_t steps = hyb::f8_steps(k), rows16 = hyb::f8_rows16(m);
  const size_t codes = size_t(rows16 / 16) * steps * hyb::kPanelStep;
  const size_t scales = (size_t((steps + 3) / 4) * rows16 * 4 + 255) / 256 * 256;
  if (x) *x = hyb_f8{base, base + codes};
  return codes + scales;
}

}  // namespace

extern "C" {

hyb_status hyb_f8_size(int64_t rows, int64_t k, size_t* code_bytes, size_t* scale_bytes) {
  const hyb_status st = check_shape(rows, k);
  if (st != HYB_OK) return st;
  if (!code_bytes || !scale_bytes) return fail(HYB_ERR_INVALID_ARG, "code_bytes or scale_bytes is NULL");
  const int64_t steps = hyb::f8_steps(k), rows16 = k > 0 ? hyb::f8_rows16(rows) : 0;
  *code_bytes = size_t(rows16 / 16) * steps * hyb::kPanelStep;
  *scale_bytes = size_t((steps + 3) / 4) * rows16 * 4;
  return ok();
}

hyb_status hyb_f8_quantize(const void* a, int32_t dtype, int64_t rows, int64_t k, int64_t lda, int32_t kind,
                           const hyb_f8* dst, void* stream) {
  if (!known_type(dtype)) return fail(HYB_ERR_DTYPE, "dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", dtype);
  if (kind != HYB_F8_WEIGHT && kind != HYB_F8_ROWS)
    return fail(HYB_ERR_INVALID_ARG, "kind %d is not HYB_F8_WEIGHT or HYB_F8_ROWS", kind);
  hyb_status st = check_shape(rows, k);
  if (st != HYB_OK) return st;
  if (rows == 0 || k == 0) return ok();
  if ((st = check_plain(a, dtype, k, lda, "a")) != HYB_OK) return st;
  if ((st = check_f8(dst, "dst")) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_f8_quantize(a, dtype, rows, k, lda, kind, *dst, static_cast<hipStream_t>(stream)),
                         "f8 quantise launch");
}

hyb_status hyb_f8_dequantize(const hyb_f8* src, int64_t rows, int64_t k, void* a, int32_t dtype, int64_t lda,
                             void* stream) {
  if (!known_type(dtype)) return fail(HYB_ERR_DTYPE, "dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", dtype);
  hyb_status st = check_shape(rows, k);
  if (st != HYB_OK) return st;
  if (rows == 0 || k == 0) return ok();
  if ((st = check_f8(src, "src")) != HYB_OK) return st;
  if ((st = check_plain(a, dtype, k, lda, "a")) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_f8_dequantize(*src, rows, k, a, dtype, lda, static_cast<hipStream_t>(stream)),
                         "f8 read-back launch");
}

hyb_status hyb_f8_gemm_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes) {
  hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (m < 0) return fail(HYB_ERR_SHAPE, "m = %d is negative", m);
  if (!bytes) return fail(HYB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (m == 0 || n == 0 || k == 0) return ok();
  *bytes = hyb::f8_workspace_bytes(n, k, m, hyb::device_cus());
  return ok();
}

hyb_status hyb_f8_gemm(const hyb_f8* w, int64_t n, int64_t k, const hyb_f8* x, int32_t m, void* y, int32_t y_dtype,
                       int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  const hyb_status st = check_gemm(w, n, k, x, m, y, y_dtype, ldy, workspace, workspace_bytes);
  if (st != HYB_OK) return st;
  if (m == 0 || n == 0) return ok();
  const hyb_f8 none{nullptr, nullptr};
  return hyb::hip_status(hyb::launch_f8_gemm(k > 0 ? *w : none, n, k, k > 0 ? *x : none, m, y, y_dtype, ldy,
                                             workspace_bytes > 0 ? static_cast<float*>(workspace) : nullptr,
                                             static_cast<hipStream_t>(stream)),
                         "f8 gemm launch");
}

hyb_status hyb_f8_linear_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes) {
  hyb_status st = hyb_f8_gemm_workspace_size(n, k, m, bytes);
  if (st != HYB_OK || m == 0 || n == 0 || k == 0) return st;
  *bytes += linear_scratch(k, m, nullptr);
  return ok();
}

hyb_status hyb_f8_linear(const hyb_f8* w, int64_t n, int64_t k, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                         void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!known_type(x_dtype)) return fail(HYB_ERR_DTYPE, "x_dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", x_dtype);
  size_t need = 0;
  hyb_status st = hyb_f8_linear_workspace_size(n, k, m, &need);
  if (st != HYB_OK) return st;
  if (workspace_bytes < need)
    return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this product needs %zu", workspace_bytes, need);
  if (m > 0 && n > 0 && k > 0) {
    if ((st = check_plain(x, x_dtype, k, ldx, "x")) != HYB_OK) return st;
    if (!workspace || !aligned(workspace, 16))
      return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  }
  hyb_f8 X{nullptr, nullptr};
  char* at = static_cast<char*>(workspace);
  const size_t used = need > 0 ? linear_scratch(k, m, &X, at) : 0;
  // the product's checks come before anything is enqueued
  if ((st = check_gemm(w, n, k, &X, m, y, y_dtype, ldy, need > used ? at + used : nullptr, need - used)) != HYB_OK)
    return st;
  if (m == 0 || n == 0) return ok();
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (hyb::f8_fused(n, k, m, y_dtype))
    return hyb::hip_status(hyb::launch_f8_fused(*w, n, k, x, x_dtype, m, ldx, y, y_dtype, ldy, s), "f8 product launch");
  if (k > 0) {
    st = hyb::hip_status(hyb::launch_f8_quantize(x, x_dtype, m, k, ldx, HYB_F8_ROWS, X, s), "f8 quantise launch");
    if (st != HYB_OK) return st;
  }
  const hyb_f8 none{nullptr, nullptr};
  return hyb::hip_status(hyb::launch_f8_gemm(k > 0 ? *w : none, n, k, X, m, y, y_dtype, ldy,
                                             need > used ? reinterpret_cast<float*>(at + used) : nullptr, s),
                         "f8 gemm launch");
}

}  // extern "C"
