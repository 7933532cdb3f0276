/*
 * hyb_gated.h -- C ABI of libhyb's gated feed-forward projection and its
 * gradients.
 *
 * For m tokens X (m x k), a gate and an up projection W_g, W_u (n x k each):
 *   G = X W_g'^T,  U = X W_u'^T,  H = act(G) * U      (elementwise)
 * and for the gradient dH (m x n) of H
 *   dU = dH * act(G),  dG = dH * U * act'(G)
 *   dX = dG W_g' + dU W_u',  dW_g = dG^T X,  dW_u = dU^T X
 * Both weights are packed tile-hybrid matrices (hyb.h; of one shape, type,
 * tile size and metadata kind, with tile maps of their own), or both 4-bit ones
 * (hyb_q4.h; no gradients).  W' is what the streams stand for: dropped entries
 * of sparse tiles are zero.
 *
 * act: HYB_ACT_SILU g / (1 + exp(-g)); HYB_ACT_GELU g Phi(g), Phi the normal
 * distribution function; HYB_ACT_GELU_TANH its usual approximation
 * g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2.
 *
 * Products are exact and summed in fp32, act is taken of the fp32 sums, and H is
 * rounded once to the 16-bit type of X.  The backward pass takes G and U in fp32
 * (rounded to 16 bits they would add as much to the gradients' errors as the
 * roundings below do); dG and dU are rounded once to the 16-bit type of its
 * products (bf16; or fp16, scaled by the power of two that brings the
 * largest finite one to [2^14, 2^15), so that they neither overflow nor, down
 * to 2^-28 of the largest, lose bits) and the gradients are summed in fp32 and
 * rounded once.
 *
 * Conventions as in hyb.h and hyb_q4.h: host checks first, work enqueued on
 * `stream`, no allocation, capturable; outputs overlap neither the inputs nor
 * each other.  The caller's workspace (device, 16-byte aligned, no initial
 * contents) holds the bytes that hyb_gated_workspace_size gives; calls that
 * overlap on one workspace race.
 */
#ifndef HYB_GATED_H_
#define HYB_GATED_H_

#include "hyb_q4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { HYB_ACT_SILU = 1, HYB_ACT_GELU = 2, HYB_ACT_GELU_TANH = 3 };

/* The two weights: layouts and streams of packed matrices with gate4 and up4
 * NULL, or gate4 and up4 (4-bit, n x k each) with the others NULL (n and k are
 * read for 4-bit ones only). */
typedef struct {
  const hyb_layout* gate_layout;
  const hyb_packed* gate;
  const hyb_layout* up_layout;
  const hyb_packed* up;
  const hyb_q4* gate4;
  const hyb_q4* up4;
  int64_t n, k;
} hyb_gated_pair;

enum { HYB_GATED_FORWARD = 0, HYB_GATED_DX = 1, HYB_GATED_DW = 2 };

/* Workspace bytes of hyb_gated (`what` = HYB_GATED_FORWARD) or
 * hyb_gated_backward (HYB_GATED_DX, HYB_GATED_DW or both) for m tokens on the
 * current device.  Host only. */
hyb_status hyb_gated_workspace_size(const hyb_gated_pair* w, int32_t m, int32_t what, size_t* bytes);

/* H.
 *   x     device m x k of x_dtype (HYB_BF16 or HYB_F16; packed weights' own
 *         type), row stride ldx >= k; for packed weights 16-byte aligned with
 *         ldx % 8 == 0 and ldx < 2^22, else element-aligned
 *   h     device m x n of x_dtype, row stride ldh >= n, element-aligned
 *   g, u  device m x n fp32, row strides ldg, ldu >= n, element-aligned:
 *         receive G and U for hyb_gated_backward; both or neither (NULL), and
 *         neither with 4-bit weights (HYB_ERR_UNSUPPORTED)
 * 0 <= m <= 2^22; 1 <= n, k <= 2^21 for packed weights, 0 <= n <= 2^27 - 16
 * and 0 <= k <= 2^22 for 4-bit ones (k = 0 gives zeros).  A launch bounds their
 * products, and what is beyond is HYB_ERR_UNSUPPORTED: for packed weights
 * ceil(n/128) ceil(m/64), ceil(k/128) ceil(m/64) and ceil(n/128) ceil(k/128) stay
 * below 2^22 (2.4 million tokens of 14336 outputs), for 4-bit ones ceil(n/128)
 * ceil(m/16) below 2^23 suffices.  Row strides of h, g, u, dh, dx, dw_gate and dw_up
 * are at most 2^31. */
hyb_status hyb_gated(const hyb_gated_pair* w, int32_t act, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                     void* h, int64_t ldh, float* g, int64_t ldg, float* u, int64_t ldu, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Gradients (packed weights; 4-bit ones are HYB_ERR_UNSUPPORTED); g and u are
 * what hyb_gated gave for the same weights, x and act.
 *   dh      device m x n of x_dtype, row stride lddh >= n, element-aligned
 *   dx      device m x k of x_dtype, row stride lddx >= k, element-aligned, or
 *           NULL
 *   dw_gate, dw_up  device n x k of x_dtype, row strides >= k,
 *           element-aligned; both or neither (NULL).  Dense: the gradient of
 *           every entry, dropped ones included. */
hyb_status hyb_gated_backward(const hyb_gated_pair* w, int32_t act, const void* x, int32_t x_dtype, int32_t m,
                              int64_t ldx, const float* g, int64_t ldg, const float* u, int64_t ldu, const void* dh,
                              int64_t lddh, void* dx, int64_t lddx, void* dw_gate, int64_t lddw_gate, void* dw_up,
                              int64_t lddw_up, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HYB_GATED_H_ */
