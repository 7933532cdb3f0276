/*
 * hyb_clip.h -- C ABI of libhyb's 2-norm over a list of tensors, and their
 * scaling by it (gradients before an optimiser's step).
 *
 *   norm  = sqrt(sum over all elements of all tensors of a^2)
 *   out   = a * min(1, max_norm / (norm + 1e-6))
 *
 * Squares are taken and summed in 64 bits, in an order that depends on the
 * tensors' sizes and strides alone; the norm is rounded once to fp32 (an
 * infinity where it lies beyond fp32), the factor is computed in 64 bits and
 * rounded to fp32, each product rounded to fp32 and then to the tensor's type.
 * A NaN anywhere makes the norm, and every element scaled, NaN; an infinity
 * makes the norm infinite and the factor 0 (and the infinities NaN), or NaN where
 * max_norm is infinite too.
 *
 * Conventions as in hyb.h: host checks first, work enqueued on `stream`, no
 * allocation, capturable.  The caller's workspace (device, 16-byte aligned, no
 * initial contents) holds hyb_clip_workspace_size bytes; calls that overlap on
 * one workspace race.
 */
#ifndef HYB_CLIP_H_
#define HYB_CLIP_H_

#include "hyb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor: rows of `cols` contiguous elements of `dtype` (HYB_F16, HYB_BF16
 * or HYB_F32) with row strides lda and ldo elements (>= cols where rows > 1), at
 * device addresses aligned to the element.  A contiguous tensor of any shape is
 * one row.  `out` may be `data` itself (with ldo = lda); else the addresses from
 * its first to its last element hold no element of another data or out of the
 * list, nor of rows between them.  0 <= rows, cols and rows * cols <= 2^40;
 * the rows reach over at most 2^44 elements. */
typedef struct {
  const void* data;
  void* out;
  int64_t rows, cols, lda, ldo;
  int32_t dtype;
} hyb_tensor;

/* Workspace bytes for `count` >= 0 tensors of these sizes, of hyb_norm or of
 * hyb_clip.  Host only.  data and out are not looked at; an ldo that hyb_clip would
 * refuse, as where a norm's tensors have no out, counts as lda. */
hyb_status hyb_clip_workspace_size(int64_t count, const hyb_tensor* tensors, size_t* bytes);

/* norm: device fp32, one element, 4-byte aligned.  `tensors` is host memory,
 * read before the call returns; `out` and `ldo` are not looked at. */
hyb_status hyb_norm(int64_t count, const hyb_tensor* tensors, float* norm, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Scales every tensor; max_norm >= 0 (not NaN).  `norm` receives the norm of
 * the data (it must not overlap them).  Tensors in place whose factor is 1 are
 * not rewritten. */
hyb_status hyb_clip(int64_t count, const hyb_tensor* tensors, float max_norm, float* norm, void* workspace,
                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HYB_CLIP_H_ */
