// Host side of the 4-bit entry points (include/hyb_q4.h): argument checks,
// then the launch.
#include "hyb_q4_internal.h"

namespace {

using hyb::fail;
using hyb::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_type(int32_t dt) { return dt == HYB_F16 || dt == HYB_BF16 || dt == HYB_F32; }

hyb_status check_shape(int64_t n, int64_t k) {
  if (n < 0 || n > hyb::kQ4MaxRows)
    return fail(HYB_ERR_SHAPE, "n = %lld outside [0, %lld]", (long long)n, (long long)hyb::kQ4MaxRows);
  if (k < 0 || k > hyb::kQ4MaxK)
    return fail(HYB_ERR_SHAPE, "k = %lld outside [0, %lld]", (long long)k, (long long)hyb::kQ4MaxK);
  return HYB_OK;
}

hyb_status check_q4(const hyb_q4* p, const char* name) {
  if (!p || !p->codes || !p->scales) return fail(HYB_ERR_INVALID_ARG, "%s, its codes or its scales are NULL", name);
  if (!aligned(p->codes, 16) || !aligned(p->scales, 16))
    return fail(HYB_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", name);
  return HYB_OK;
}

hyb_status check_plain(const void* a, int32_t dtype, int64_t k, int64_t ld, const char* name) {
  if (!a || !aligned(a, dtype == HYB_F32 ? 4 : 2))
    return fail(HYB_ERR_INVALID_ARG, "%s is NULL or not aligned to its element size", name);
  if (ld < k) return fail(HYB_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)ld, (long long)k);
  if (ld > (int64_t(1) << 31))
    return fail(HYB_ERR_UNSUPPORTED, "%s row stride %lld is above 2^31", name, (long long)ld);
  return HYB_OK;
}

}  // namespace

extern "C" {

hyb_status hyb_q4_size(int64_t n, int64_t k, size_t* code_bytes, size_t* scale_bytes) {
  const hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (!code_bytes || !scale_bytes) return fail(HYB_ERR_INVALID_ARG, "code_bytes or scale_bytes is NULL");
  const int64_t rows16 = k > 0 ? hyb::q4_rows16(n) : 0;
  *code_bytes = size_t(rows16 / 16) * hyb::q4_steps(k) * hyb::kQ4StepBytes;
  *scale_bytes = size_t(rows16) * (hyb::q4_quads(k) * 16 + 1);
  return ok();
}

hyb_status hyb_q4_quantize(const void* a, int32_t dtype, int64_t n, int64_t k, int64_t lda, const hyb_q4* dst,
                           void* stream) {
  if (!known_type(dtype)) return fail(HYB_ERR_DTYPE, "dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", dtype);
  hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (n == 0 || k == 0) return ok();
  if ((st = check_plain(a, dtype, k, lda, "a")) != HYB_OK) return st;
  if ((st = check_q4(dst, "dst")) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_q4_quantize(a, dtype, n, k, lda, *dst, static_cast<hipStream_t>(stream)),
                         "q4 quantise launch");
}

hyb_status hyb_q4_dequantize(const hyb_q4* src, int64_t n, int64_t k, void* a, int32_t dtype, int64_t lda,
                             void* stream) {
  if (!known_type(dtype)) return fail(HYB_ERR_DTYPE, "dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", dtype);
  hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (n == 0 || k == 0) return ok();
  if ((st = check_q4(src, "src")) != HYB_OK) return st;
  if ((st = check_plain(a, dtype, k, lda, "a")) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_q4_dequantize(*src, n, k, a, dtype, lda, static_cast<hipStream_t>(stream)),
                         "q4 read-back launch");
}

hyb_status hyb_q4_gemm_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes) {
  const hyb_status st = check_shape(n, k);
  if (st != HYB_OK) return st;
  if (m < 0 || m > hyb::kQ4MaxTokens) return fail(HYB_ERR_SHAPE, "m = %d outside [0, %d]", m, hyb::kQ4MaxTokens);
  if (!bytes) return fail(HYB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (m == 0 || n == 0 || k == 0) return ok();
  const hyb::Q4Route r = hyb::q4_route(n, k, m, 1, hyb::device_cus());
  *bytes = hyb::q4_pack_bytes(r, k, m) + hyb::q4_part_bytes(r, n, m, 1);
  return ok();
}

hyb_status hyb_q4_gemm(const hyb_q4* w, int64_t n, int64_t k, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                       void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (x_dtype != HYB_F16 && x_dtype != HYB_BF16)
    return fail(HYB_ERR_DTYPE, "x_dtype %d is not HYB_F16 or HYB_BF16", x_dtype);
  if (!known_type(y_dtype)) return fail(HYB_ERR_DTYPE, "y_dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", y_dtype);
  size_t need = 0;
  hyb_status st = hyb_q4_gemm_workspace_size(n, k, m, &need);
  if (st != HYB_OK) return st;
  if (workspace_bytes < need)
    return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this product needs %zu", workspace_bytes, need);
  if (need > 0 && (!workspace || !aligned(workspace, 16)))
    return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  if (m == 0 || n == 0) return ok();
  if ((st = check_plain(y, y_dtype, n, ldy, "y")) != HYB_OK) return st;
  if (k > 0) {
    if ((st = check_q4(w, "w")) != HYB_OK) return st;
    if ((st = check_plain(x, x_dtype, k, ldx, "x")) != HYB_OK) return st;
    const hyb::Q4Route r = hyb::q4_route(n, k, m, 1, hyb::device_cus());
    if (hyb::q4_groups(r, n, m, 1) >= hyb::kQ4MaxTiles)
      return fail(HYB_ERR_UNSUPPORTED, "n x m = %lld x %d is too large for one launch", (long long)n, m);
  }
  const hyb_q4 none{nullptr, nullptr};
  return hyb::hip_status(hyb::launch_q4_product(k > 0 ? *w : none, nullptr, 0, n, k, x, x_dtype, m, ldx, y, y_dtype,
                                                ldy, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)),
                         "q4 product launch");
}

}  // extern "C"
