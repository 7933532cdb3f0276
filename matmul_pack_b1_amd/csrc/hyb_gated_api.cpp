// Host side of the gated projection (include/hyb_gated.h): argument checks,
// then the launches.
#include "hyb_gated_internal.h"
#include "hyb_q4_internal.h"

namespace {

using hyb::fail;
using hyb::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

hyb_status check_streams(const hyb_layout& L, const hyb_packed* P, const char* name) {
  if (!P) return fail(HYB_ERR_INVALID_ARG, "%s streams are NULL", name);
  if ((L.dense_bytes > 0 && (!P->dense || !aligned(P->dense, 16))) ||
      (L.val_bytes > 0 && (!P->val || !aligned(P->val, 16))) ||
      (L.meta_bytes > 0 && (!P->meta || !aligned(P->meta, 16))) ||
      (L.tidx_bytes > 0 && (!P->tidx || !aligned(P->tidx, 4))))
    return fail(HYB_ERR_INVALID_ARG, "a %s stream is NULL or misaligned", name);
  return HYB_OK;
}

// The pair's shape and type; `streams`: its device addresses too.  *dtype is 0
// for 4-bit weights.
hyb_status check_pair(const hyb_gated_pair* w, bool streams, int64_t* n, int64_t* k, int32_t* dtype) {
  if (!w) return fail(HYB_ERR_INVALID_ARG, "the weights are NULL");
  const bool packed = w->gate_layout || w->up_layout || w->gate || w->up, four = w->gate4 || w->up4;
  if (packed == four) return fail(HYB_ERR_INVALID_ARG, "the weights are either two packed ones or two 4-bit ones");
  if (four) {
    if (!w->gate4 || !w->up4) return fail(HYB_ERR_INVALID_ARG, "one of the 4-bit weights is NULL");
    *n = w->n;
    *k = w->k;
    *dtype = 0;
    size_t a, b;
    const hyb_status st = hyb_q4_size(*n, *k, &a, &b);
    if (st != HYB_OK) return st;
    for (const hyb_q4* p : {w->gate4, w->up4})
      if (streams && *n > 0 && *k > 0 &&
          (!p->codes || !p->scales || !aligned(p->codes, 16) || !aligned(p->scales, 16)))
        return fail(HYB_ERR_INVALID_ARG, "codes or scales are NULL or not 16-byte aligned");
    return HYB_OK;
  }
  if (!w->gate_layout || !w->up_layout) return fail(HYB_ERR_INVALID_ARG, "one of the layouts is NULL");
  for (const hyb_layout* l : {w->gate_layout, w->up_layout}) {
    const hyb_status st = hyb_layout_check(l);
    if (st != HYB_OK) return st;
  }
  const hyb_layout &G = *w->gate_layout, &U = *w->up_layout;
  auto device_tile = [](int32_t b) { return b == 64 || b == 128 || b == 256; };
  if (!device_tile(G.b1) || !device_tile(G.b2))
    return fail(HYB_ERR_UNSUPPORTED, "tile %dx%d: sides must be 64, 128 or 256", G.b1, G.b2);
  if (G.n != U.n || G.k != U.k)
    return fail(HYB_ERR_SHAPE, "gate is %lld x %lld, up %lld x %lld", (long long)G.n, (long long)G.k, (long long)U.n,
                (long long)U.k);
  if (G.dtype != U.dtype) return fail(HYB_ERR_DTYPE, "gate has type %d, up %d", G.dtype, U.dtype);
  if (G.b1 != U.b1 || G.b2 != U.b2 || G.meta != U.meta)
    return fail(HYB_ERR_UNSUPPORTED, "gate and up differ in tile size or metadata kind");
  *n = G.n;
  *k = G.k;
  *dtype = G.dtype;
  if (*n < 1 || *n > hyb::kGatedMaxSide || *k < 1 || *k > hyb::kGatedMaxSide)
    return fail(HYB_ERR_SHAPE, "weights %lld x %lld: need 1 <= n, k <= 2^21", (long long)*n, (long long)*k);
  if (!streams) return HYB_OK;
  const hyb_status st = check_streams(G, w->gate, "gate");
  return st != HYB_OK ? st : check_streams(U, w->up, "up");
}

hyb_status check_tokens(int32_t m) {
  return m < 0 || m > hyb::kGatedMaxTokens ? fail(HYB_ERR_SHAPE, "m = %d outside [0, %d]", m, hyb::kGatedMaxTokens) : HYB_OK;
}

hyb_status check_type(int32_t x_dtype, int32_t dtype, int32_t act) {
  if (act != HYB_ACT_SILU && act != HYB_ACT_GELU && act != HYB_ACT_GELU_TANH)
    return fail(HYB_ERR_INVALID_ARG, "act %d is not HYB_ACT_SILU, HYB_ACT_GELU or HYB_ACT_GELU_TANH", act);
  if (x_dtype != HYB_BF16 && x_dtype != HYB_F16)
    return fail(HYB_ERR_DTYPE, "x_dtype %d is not HYB_BF16 or HYB_F16", x_dtype);
  if (dtype != 0 && x_dtype != dtype)
    return fail(HYB_ERR_DTYPE, "x_dtype %d differs from the weights' type %d", x_dtype, dtype);
  return HYB_OK;
}

hyb_status check_x(const void* x, int64_t k, int64_t ldx, bool packed) {
  const uintptr_t align = packed ? 16 : 2;
  if (!x || !aligned(x, align)) return fail(HYB_ERR_INVALID_ARG, "x is NULL or not %d-byte aligned", int(align));
  if (ldx < k || (packed && ldx % 8 != 0))
    return fail(HYB_ERR_INVALID_ARG, "x row stride %lld must be >= k%s", (long long)ldx,
                packed ? " and a multiple of 8" : "");
  // the decode and matrix-core products of hyb.h address a tile of x in 32 bits
  if (ldx >= (packed ? int64_t(1) << 22 : (int64_t(1) << 31) + 1))
    return fail(HYB_ERR_UNSUPPORTED, "x row stride %lld is too large", (long long)ldx);
  return HYB_OK;
}

// A matrix of rows of `cols` elements of `size` bytes.
hyb_status check_rows(const void* p, int64_t cols, int64_t ld, const char* name, int size = 2) {
  if (!p || !aligned(p, size)) return fail(HYB_ERR_INVALID_ARG, "%s is NULL or not %d-byte aligned", name, size);
  if (ld < cols) return fail(HYB_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)ld, (long long)cols);
  if (ld > (int64_t(1) << 31))
    return fail(HYB_ERR_UNSUPPORTED, "%s row stride %lld is above 2^31", name, (long long)ld);
  return HYB_OK;
}

hyb_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (bytes < need) return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this call needs %zu", bytes, need);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  return HYB_OK;
}

// Tiles of any launch (G and U, dX, dW) stay below 2^32 threads in one grid
// dimension, and the elementwise kernels' rows too.
hyb_status check_launch(int64_t n, int64_t k, int64_t m) {
  const int64_t tn = (n + 127) / 128, tk = (k + 127) / 128, tm = (m + 63) / 64, most = int64_t(1) << 22;
  if (tn * tm >= most || tk * tm >= most || tn * tk >= most)
    return fail(HYB_ERR_UNSUPPORTED, "n x k x m = %lld x %lld x %lld is too large for one launch", (long long)n,
                (long long)k, (long long)m);
  return HYB_OK;
}

}  // namespace

extern "C" {

hyb_status hyb_gated_workspace_size(const hyb_gated_pair* w, int32_t m, int32_t what, size_t* bytes) {
  int64_t n, k;
  int32_t dtype;
  hyb_status st = check_pair(w, false, &n, &k, &dtype);
  if (st != HYB_OK) return st;
  if ((st = check_tokens(m)) != HYB_OK) return st;
  if (what < 0 || what > 3) return fail(HYB_ERR_INVALID_ARG, "what = %d", what);
  if (dtype == 0 && what != HYB_GATED_FORWARD) return fail(HYB_ERR_UNSUPPORTED, "4-bit weights have no gradients");
  if (!bytes) return fail(HYB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  if (m == 0 || n == 0 || k == 0) return ok();
  if (dtype == 0) {
    const hyb::Q4Route r = hyb::q4_route(n, k, m, 2, hyb::device_cus());
    *bytes = hyb::q4_pack_bytes(r, k, m) + hyb::q4_part_bytes(r, n, m, 2);
  } else {
    *bytes = hyb::gated_plan(*w, m, what, hyb::device_cus()).total;
  }
  return ok();
}

hyb_status hyb_gated(const hyb_gated_pair* w, int32_t act, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                     void* h, int64_t ldh, float* g, int64_t ldg, float* u, int64_t ldu, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int64_t n, k;
  int32_t dtype;
  hyb_status st = check_pair(w, true, &n, &k, &dtype);
  if (st != HYB_OK) return st;
  if ((st = check_type(x_dtype, dtype, act)) != HYB_OK) return st;
  if ((st = check_tokens(m)) != HYB_OK) return st;
  if ((g == nullptr) != (u == nullptr)) return fail(HYB_ERR_INVALID_ARG, "one of g and u is NULL");
  if (dtype == 0 && g) return fail(HYB_ERR_UNSUPPORTED, "4-bit weights have no gradients: g and u must be NULL");
  size_t need = 0;
  if ((st = hyb_gated_workspace_size(w, m, HYB_GATED_FORWARD, &need)) != HYB_OK) return st;
  if (m == 0 || n == 0) return ok();
  if ((st = check_rows(h, n, ldh, "h")) != HYB_OK) return st;
  if (g) {
    if ((st = check_rows(g, n, ldg, "g", 4)) != HYB_OK) return st;
    if ((st = check_rows(u, n, ldu, "u", 4)) != HYB_OK) return st;
    if (g == u) return fail(HYB_ERR_INVALID_ARG, "g and u are one buffer");
  }
  if (k > 0 && (st = check_x(x, k, ldx, dtype != 0)) != HYB_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, need)) != HYB_OK) return st;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == 0) {
    if (k > 0 && hyb::q4_groups(hyb::q4_route(n, k, m, 2, hyb::device_cus()), n, m, 2) >= hyb::kQ4MaxTiles)
      return fail(HYB_ERR_UNSUPPORTED, "n x m = %lld x %d is too large for one launch", (long long)n, m);
    return hyb::hip_status(
        hyb::launch_q4_product(*w->gate4, w->up4, act, n, k, x, x_dtype, m, ldx, h, x_dtype, ldh, ws, s),
        "gated 4-bit launch");
  }
  if ((st = check_launch(n, k, m)) != HYB_OK) return st;
  const hyb::GatedPlan p = hyb::gated_plan(*w, m, HYB_GATED_FORWARD, hyb::device_cus());
  const hyb::GatedForward out{h, g, u, ldh, ldg, ldu};
  return hyb::hip_status(hyb::launch_gated(*w, p, act, x, x_dtype, ldx, out, ws, s), "gated launch");
}

hyb_status hyb_gated_backward(const hyb_gated_pair* w, int32_t act, const void* x, int32_t x_dtype, int32_t m,
                              int64_t ldx, const float* g, int64_t ldg, const float* u, int64_t ldu, const void* dh,
                              int64_t lddh, void* dx, int64_t lddx, void* dw_gate, int64_t lddw_gate, void* dw_up,
                              int64_t lddw_up, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t n, k;
  int32_t dtype;
  hyb_status st = check_pair(w, true, &n, &k, &dtype);
  if (st != HYB_OK) return st;
  if (dtype == 0) return fail(HYB_ERR_UNSUPPORTED, "4-bit weights have no gradients");
  if ((st = check_type(x_dtype, dtype, act)) != HYB_OK) return st;
  if ((st = check_tokens(m)) != HYB_OK) return st;
  if ((dw_gate == nullptr) != (dw_up == nullptr)) return fail(HYB_ERR_INVALID_ARG, "one of dw_gate and dw_up is NULL");
  const int what = (dx ? HYB_GATED_DX : 0) | (dw_gate ? HYB_GATED_DW : 0);
  if (what == 0) return ok();
  if (dw_gate) {
    if ((st = check_rows(dw_gate, k, lddw_gate, "dw_gate")) != HYB_OK) return st;
    if ((st = check_rows(dw_up, k, lddw_up, "dw_up")) != HYB_OK) return st;
    if (dw_gate == dw_up) return fail(HYB_ERR_INVALID_ARG, "dw_gate and dw_up are one buffer");
  }
  size_t need = 0;
  if ((st = hyb_gated_workspace_size(w, m, what, &need)) != HYB_OK) return st;
  if (m > 0) {
    if ((st = check_x(x, k, ldx, true)) != HYB_OK) return st;
    if ((st = check_rows(g, n, ldg, "g", 4)) != HYB_OK) return st;
    if ((st = check_rows(u, n, ldu, "u", 4)) != HYB_OK) return st;
    if ((st = check_rows(dh, n, lddh, "dh")) != HYB_OK) return st;
    if (dx && (st = check_rows(dx, k, lddx, "dx")) != HYB_OK) return st;
    if ((st = check_ws(workspace, workspace_bytes, need)) != HYB_OK) return st;
  } else if (!dw_gate) {
    return ok();
  }
  if ((st = check_launch(n, k, m)) != HYB_OK) return st;
  const hyb::GatedPlan p = hyb::gated_plan(*w, m, what, hyb::device_cus());
  const hyb::GatedBackward b{g, u, dh, ldg, ldu, lddh, dx, lddx, {dw_gate, dw_up}, {lddw_gate, lddw_up}};
  return hyb::hip_status(
      hyb::launch_gated_backward(*w, p, act, x, x_dtype, ldx, b, static_cast<char*>(workspace),
                                 static_cast<hipStream_t>(stream)),
      "gated backward launch");
}

}  // extern "C"
