// Host side of the cross entropy (include/hyb_xent.h): argument checks, then
// the launches.
#include "hyb_xent_internal.h"

namespace {

using hyb::fail;
using hyb::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Largest rows x k the kernels' 32-bit panel and tile numbers cover.
constexpr int64_t kMaxVocab = hyb::kF8MaxRows;
constexpr int32_t kMaxTokens = 1 << 22;
constexpr int64_t kMaxK = int64_t(1) << 21;

hyb_status check_head(const hyb_head* h, bool streams) {
  if (!h) return fail(HYB_ERR_INVALID_ARG, "head is NULL");
  if ((h->f8 != nullptr) == (h->layout != nullptr))
    return fail(HYB_ERR_INVALID_ARG, "a head is either packed (layout) or 8-bit (f8)");
  int64_t n, k;
  if (h->f8) {
    if (h->packed) return fail(HYB_ERR_INVALID_ARG, "an 8-bit head has no packed streams");
    n = h->n;
    k = h->k;
    if (n < 0 || k < 0)
      return fail(HYB_ERR_SHAPE, "head %lld x %lld", (long long)n, (long long)k);
    if (streams && n > 0 && k > 0 &&
        (!h->f8->codes || !h->f8->scales || !aligned(h->f8->codes, 16) || !aligned(h->f8->scales, 16)))
      return fail(HYB_ERR_INVALID_ARG, "head codes or scales are NULL or not 16-byte aligned");
  } else {
    hyb_status st = hyb_layout_check(h->layout);
    if (st != HYB_OK) return st;
    const hyb_layout& L = *h->layout;
    auto device_tile = [](int32_t b) { return b == 64 || b == 128 || b == 256; };
    if (!device_tile(L.b1) || !device_tile(L.b2))
      return fail(HYB_ERR_UNSUPPORTED, "tile %dx%d: sides must be 64, 128 or 256", L.b1, L.b2);
    n = L.n;
    k = L.k;
    if (streams) {
      const hyb_packed* P = h->packed;
      if (!P) return fail(HYB_ERR_INVALID_ARG, "head streams are NULL");
      if ((L.dense_bytes > 0 && (!P->dense || !aligned(P->dense, 16))) ||
          (L.val_bytes > 0 && (!P->val || !aligned(P->val, 16))) ||
          (L.meta_bytes > 0 && (!P->meta || !aligned(P->meta, 16))) ||
          (L.tidx_bytes > 0 && (!P->tidx || !aligned(P->tidx, 4))))
        return fail(HYB_ERR_INVALID_ARG, "a head stream is NULL or misaligned");
    }
  }
  if (n < 1 || n > kMaxVocab || k < 1 || k > kMaxK)
    return fail(HYB_ERR_SHAPE, "head %lld x %lld: need 1 <= n <= 2^27 - 16 and 1 <= k <= 2^21", (long long)n, (long long)k);
  return HYB_OK;
}

hyb_status check_call(const hyb_head* h, int64_t n_vocab, const void* x, int32_t dt, int32_t m, int64_t ldx,
                      const int64_t* target) {
  hyb_status st = check_head(h, true);
  if (st != HYB_OK) return st;
  const int64_t n = h->f8 ? h->n : h->layout->n, k = h->f8 ? h->k : h->layout->k;
  if (n_vocab < 1 || n_vocab > n)
    return fail(HYB_ERR_SHAPE, "n_vocab = %lld outside [1, %lld]", (long long)n_vocab, (long long)n);
  if (dt != HYB_BF16 && dt != HYB_F16) return fail(HYB_ERR_DTYPE, "x_dtype %d is not HYB_BF16 or HYB_F16", dt);
  if (h->layout && dt != h->layout->dtype)
    return fail(HYB_ERR_DTYPE, "x_dtype %d differs from the head's type %d", dt, h->layout->dtype);
  if (m < 0 || m > kMaxTokens) return fail(HYB_ERR_SHAPE, "m = %d outside [0, %d]", m, kMaxTokens);
  if ((n + 255) / 256 * ((int64_t(m) + 63) / 64) >= (int64_t(1) << 23))
    return fail(HYB_ERR_UNSUPPORTED, "n x m = %lld x %d is too large for one launch", (long long)n, m);
  if (m == 0) return HYB_OK;
  const uintptr_t align = h->f8 ? 2 : 16;
  if (!x || !aligned(x, align)) return fail(HYB_ERR_INVALID_ARG, "x is NULL or not %d-byte aligned", int(align));
  if (ldx < k || (!h->f8 && ldx % 8 != 0))
    return fail(HYB_ERR_INVALID_ARG, "x row stride %lld must be >= k%s", (long long)ldx,
                h->f8 ? "" : " and a multiple of 8");
  // the decode and matrix-core products of hyb.h address a tile of x in 32 bits
  if (ldx >= (int64_t(1) << 22)) return fail(HYB_ERR_UNSUPPORTED, "x row stride %lld must be below 2^22", (long long)ldx);
  if (!target || !aligned(target, 8)) return fail(HYB_ERR_INVALID_ARG, "target is NULL or not 8-byte aligned");
  return HYB_OK;
}

hyb_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (bytes < need) return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this call needs %zu", bytes, need);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  return HYB_OK;
}

}  // namespace

extern "C" {

hyb_status hyb_xent_workspace_size(const hyb_head* head, int32_t m, int32_t what, size_t* bytes) {
  hyb_status st = check_head(head, false);
  if (st != HYB_OK) return st;
  if (m < 0 || m > kMaxTokens) return fail(HYB_ERR_SHAPE, "m = %d outside [0, %d]", m, kMaxTokens);
  if (what < 0 || what > 3) return fail(HYB_ERR_INVALID_ARG, "what = %d", what);
  if ((what & HYB_XENT_DW) && head->f8) return fail(HYB_ERR_UNSUPPORTED, "an 8-bit head has no weight gradient");
  if (!bytes) return fail(HYB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = m == 0 ? 0 : hyb::xent_plan(*head, m, what, hyb::device_cus()).total;
  return ok();
}

hyb_status hyb_xent_piece_rows(const hyb_head* head, int32_t m, int32_t what, int64_t* rows) {
  hyb_status st = check_head(head, false);
  if (st != HYB_OK) return st;
  if (m < 1 || m > kMaxTokens) return fail(HYB_ERR_SHAPE, "m = %d outside [1, %d]", m, kMaxTokens);
  if (what < 0 || what > 3) return fail(HYB_ERR_INVALID_ARG, "what = %d", what);
  if ((what & HYB_XENT_DW) && head->f8) return fail(HYB_ERR_UNSUPPORTED, "an 8-bit head has no weight gradient");
  if (!rows) return fail(HYB_ERR_INVALID_ARG, "rows is NULL");
  *rows = hyb::xent_plan(*head, m, what, hyb::device_cus()).at_once;
  return ok();
}

hyb_status hyb_xent(const hyb_head* head, int64_t n_vocab, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                    const int64_t* target, int64_t ignore_index, float* loss, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  hyb_status st = check_call(head, n_vocab, x, x_dtype, m, ldx, target);
  if (st != HYB_OK) return st;
  if (m == 0) return ok();
  if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4))
    return fail(HYB_ERR_INVALID_ARG, "loss or lse is NULL or misaligned");
  const hyb::XentPlan p = hyb::xent_plan(*head, m, HYB_XENT_LOSS, hyb::device_cus());
  if ((st = check_ws(workspace, workspace_bytes, p.total)) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_xent(*head, p, n_vocab, x, x_dtype, ldx, target, ignore_index, loss, lse,
                                          static_cast<char*>(workspace), static_cast<hipStream_t>(stream)),
                         "cross entropy launch");
}

hyb_status hyb_xent_backward(const hyb_head* head, int64_t n_vocab, const void* x, int32_t x_dtype, int32_t m,
                             int64_t ldx, const int64_t* target, int64_t ignore_index, const float* lse,
                             const float* grad, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                             size_t workspace_bytes, void* stream) {
  hyb_status st = check_call(head, n_vocab, x, x_dtype, m, ldx, target);
  if (st != HYB_OK) return st;
  const int64_t k = head->f8 ? head->k : head->layout->k;
  if (dw && head->f8) return fail(HYB_ERR_UNSUPPORTED, "an 8-bit head has no weight gradient");
  if (dw && (!aligned(dw, 2) || lddw < k))
    return fail(HYB_ERR_INVALID_ARG, "dw is misaligned or its row stride %lld is below k", (long long)lddw);
  if (m > 0 && dx && (!aligned(dx, 2) || lddx < k))
    return fail(HYB_ERR_INVALID_ARG, "dx is misaligned or its row stride %lld is below k", (long long)lddx);
  if ((dx && lddx > (int64_t(1) << 31)) || (dw && lddw > (int64_t(1) << 31)))
    return fail(HYB_ERR_UNSUPPORTED, "a row stride is above 2^31");
  if (!dx && !dw) return ok();
  if (m == 0 && !dw) return ok();
  if (m > 0 && (!lse || !grad || !aligned(lse, 4) || !aligned(grad, 4)))
    return fail(HYB_ERR_INVALID_ARG, "lse or grad is NULL or misaligned");
  const int what = (dx ? HYB_XENT_DX : 0) | (dw ? HYB_XENT_DW : 0);
  const hyb::XentPlan p = hyb::xent_plan(*head, m, what, hyb::device_cus());
  if ((st = check_ws(workspace, workspace_bytes, m == 0 ? 0 : p.total)) != HYB_OK) return st;
  return hyb::hip_status(hyb::launch_xent_backward(*head, p, n_vocab, x, x_dtype, ldx, target, ignore_index, lse, grad,
                                                   dx, lddx, dw, lddw, static_cast<char*>(workspace),
                                                   static_cast<hipStream_t>(stream)),
                         "cross entropy backward launch");
}

}  // extern "C"
