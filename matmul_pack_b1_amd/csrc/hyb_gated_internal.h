// Internal interface between the host-side checks of the gated projection
// (hyb_gated_api.cpp) and its kernels (hyb_gated.hip).  Everything reaching a
// launcher has been validated.
#pragma once

#include "../../include/hyb_gated.h"
#include "hyb_internal.h"

namespace hyb {

// Largest n, k of packed weights: 16 panels' steps stay within 32 bits.
constexpr int64_t kGatedMaxSide = int64_t(1) << 21;
constexpr int32_t kGatedMaxTokens = 1 << 22;

// One call over packed weights: how it runs, and where its buffers lie in the
// workspace (byte offsets).
struct GatedPlan {
  int64_t n, k, m, m16, m64;
  bool decode;   // forward: the gated decode kernel ...
  bool rows;     // ... or G and U as fp32 in memory, then act ...
  bool grouped;  // ... from the grouped decode kernel, or the matrix-core ones
  int bp;       // token panels per tile
  bool small_dw;  // dW in tiles of 128 x 128
  bool both;      // dX and dW in one launch
  int64_t whole;  // forward tiles that run over all of k; the others are cut
  int parts;      // parts of those, or cuts of n in the dX product
  size_t x, w[2], g[2], gu, split, split_bytes, dx, misc, total;
};
GatedPlan gated_plan(const hyb_gated_pair& w, int64_t m, int what, int64_t cus);

struct GatedForward {
  void* h;
  float* g;
  float* u;
  int64_t ldh, ldg, ldu;
};
hipError_t launch_gated(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int dtype, int64_t ldx,
                        const GatedForward& out, char* ws, hipStream_t s);

struct GatedBackward {
  const float* g;
  const float* u;
  const void* dh;
  int64_t ldg, ldu, lddh;
  void* dx;
  int64_t lddx;
  void* dw[2];
  int64_t lddw[2];
};
hipError_t launch_gated_backward(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int dtype,
                                 int64_t ldx, const GatedBackward& b, char* ws, hipStream_t s);

}  // namespace hyb
