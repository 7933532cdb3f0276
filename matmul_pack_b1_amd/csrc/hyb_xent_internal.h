// Internal interface between the host-side checks of the cross entropy
// (hyb_xent_api.cpp) and its kernels (hyb_xent.hip).  Everything reaching a
// launcher has been validated.
#pragma once

#include "../../include/hyb_xent.h"
#include "hyb_f8_internal.h"

namespace hyb {

// One call: its shape, how the vocabulary is cut, and where its buffers lie
// in the workspace (byte offsets; 0 bytes where a buffer is not used).
struct XentPlan {
  bool f8;
  int64_t n, k;        // head
  int64_t m;           // tokens
  int64_t steps;       // steps of k in the logits product
  int64_t ksteps16;    // 64-column steps of k in 16-bit panels
  int64_t piece;       // vocabulary rows per piece of dz or of expanded tiles (multiple of 256)
  int64_t m16, m64;    // tokens rounded up
  int bp;              // token panels per tile of the logits product
  bool rows;           // few tokens or tiles: logits through the library's product
  int64_t at_once;     // vocabulary rows the call works through at a time
  int64_t chunks;      // partial softmax sums per token
  int parts;           // cuts of the vocabulary in the dX product
  size_t x, xs, part, zt, logits, w, g, dx, misc, total;
};
XentPlan xent_plan(const hyb_head& head, int64_t m, int what, int64_t cus);

hipError_t launch_xent(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int dtype, int64_t ldx,
                       const int64_t* target, int64_t ignore, float* loss, float* lse, char* ws, hipStream_t s);
hipError_t launch_xent_backward(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int dtype,
                                int64_t ldx, const int64_t* target, int64_t ignore, const float* lse,
                                const float* grad, void* dx, int64_t lddx, void* dw, int64_t lddw, char* ws,
                                hipStream_t s);

}  // namespace hyb
