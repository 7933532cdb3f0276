/*
 * hyb_xent.h -- C ABI of libhyb's softmax cross entropy over a vocabulary
 * projection, without the logits in memory.
 *
 * A head is the projection to the vocabulary, W (n x k, one row per entry),
 * held either as a packed tile-hybrid matrix (hyb.h) or as an 8-bit
 * block-scaled weight (hyb_f8.h).  For the m hidden states X (m x k):
 *   z[t, v]  = X[t, :] . W'[v, :]              v < n_vocab
 *   lse[t]   = log sum_v exp z[t, v]
 *   loss[t]  = lse[t] - z[t, target[t]]
 * and for the gradient grad[t] of loss[t]
 *   dz[t, v] = grad[t] (exp(z[t, v] - lse[t]) - [v == target[t]])
 *   dX       = dz W',   dW = dz^T X
 * W' is what the head stands for (dropped entries of 2:4 tiles are zero; an
 * 8-bit head takes X quantised per 1 x 128 block, as its product does, and
 * its dX passes through that rounding unchanged).
 *
 * Rows n_vocab .. n-1 of the head are padding: no logit, no gradient, and
 * their values are not looked at (dW is zero there).  n_vocab may be any
 * number in [1, n].  A token whose target is ignore_index counts for
 * nothing: loss, lse and its row of dX are zero and its x and grad are not
 * looked at (they may be NaN).  A target that is neither ignore_index nor in
 * [0, n_vocab) makes that token's loss and dX row, and dW, NaN.
 *
 * Products are exact and summed in fp32, softmax sums are fp32.  In the
 * backward pass dz is rounded once to the 16-bit type of the products (bf16;
 * or fp16, scaled by 2^14 over the largest |grad| rounded up to a power of two,
 * so that a dz of 4e-9 of that grad keeps 11 bits) and both gradients are
 * summed in fp32 and rounded once.  An fp16 dX over an 8-bit head takes W'
 * scaled into fp16's range: exact for blocks whose scale is within 2^21 of the
 * head's largest, off by at most 2^-31 of that largest scale for others (2^-38
 * of the largest magnitude); in bf16 all of W' is exact from 2^-126 on.
 * The vocabulary is worked through in pieces; the logits of a piece live in
 * registers (or, for few tokens, in the workspace).
 *
 * Conventions as in hyb.h and hyb_f8.h: host checks first, work enqueued on
 * `stream`, no allocation, capturable.  The caller's workspace (16-byte
 * aligned, no initial contents) holds hyb_xent_workspace_size bytes; calls
 * that overlap on one workspace race.
 */
#ifndef HYB_XENT_H_
#define HYB_XENT_H_

#include "hyb_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A head: `layout` and `packed` of a packed matrix with `f8` NULL, or `f8`
 * (a HYB_F8_WEIGHT matrix, n x k) with `layout` and `packed` NULL (n and k
 * are read for an 8-bit head only). */
typedef struct {
  const hyb_layout* layout;
  const hyb_packed* packed;
  const hyb_f8* f8;
  int64_t n, k;
} hyb_head;

enum { HYB_XENT_LOSS = 0, HYB_XENT_DX = 1, HYB_XENT_DW = 2 };

/* Workspace bytes of hyb_xent (`what` = HYB_XENT_LOSS) or hyb_xent_backward
 * (HYB_XENT_DX, HYB_XENT_DW or both) for m tokens on the current device.
 * Host only. */
hyb_status hyb_xent_workspace_size(const hyb_head* head, int32_t m, int32_t what, size_t* bytes);

/* Vocabulary rows that the call of hyb_xent_workspace_size's arguments works
 * through at a time on the current device (n: all at once; the last piece may
 * be shorter).  Host only. */
hyb_status hyb_xent_piece_rows(const hyb_head* head, int32_t m, int32_t what, int64_t* rows);

/* loss (m fp32) and lse (m fp32).
 *   x       device m x k of x_dtype (HYB_BF16 or HYB_F16; a packed head's own
 *           type), row stride ldx, k <= ldx < 2^22; 16-byte aligned with
 *           ldx % 8 == 0 for a packed head, element-aligned for an 8-bit one
 *   target  device int64[m]
 * 0 <= m <= 2^22 tokens; a head has 1 <= n <= 2^27 - 16 and
 * 1 <= k <= 2^21. */
hyb_status hyb_xent(const hyb_head* head, int64_t n_vocab, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                    const int64_t* target, int64_t ignore_index, float* loss, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Gradients; lse is what hyb_xent gave for the same head, x and n_vocab.
 *   grad  device fp32[m], the gradient of each token's loss
 *   dx    device m x k of x_dtype, row stride lddx >= k, or NULL
 *   dw    device n x k of the packed head's type, row stride lddw >= k, or
 *         NULL; dense: the gradient of every entry of W, dropped ones
 *         included.  An 8-bit head has none (HYB_ERR_UNSUPPORTED). */
hyb_status hyb_xent_backward(const hyb_head* head, int64_t n_vocab, const void* x, int32_t x_dtype, int32_t m,
                             int64_t ldx, const int64_t* target, int64_t ignore_index, const float* lse,
                             const float* grad, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                             size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HYB_XENT_H_ */
