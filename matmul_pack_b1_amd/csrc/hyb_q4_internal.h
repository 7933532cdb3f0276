// Internal interface between the host-side checks of the 4-bit entry points
// (hyb_q4_api.cpp, hyb_gated_api.cpp) and their kernels (hyb_q4.hip).
// Everything reaching a launcher has been validated.
#pragma once

#include "../../include/hyb_q4.h"
#include "hyb_internal.h"

namespace hyb {

// Columns of one step, and its bytes per 16-row panel.
constexpr int64_t kQ4Step = 128;
constexpr int64_t kQ4StepBytes = 1024;
constexpr int64_t kQ4MaxK = int64_t(1) << 22;
// Launch limits: 512 threads per panel, or per tile, stay below 2^32 in one
// grid dimension.
constexpr int64_t kQ4MaxRows = (int64_t(1) << 27) - 16;
constexpr int64_t kQ4MaxTiles = int64_t(1) << 23;
constexpr int32_t kQ4MaxTokens = 1 << 22;

inline int64_t q4_steps(int64_t k) { return (k + kQ4Step - 1) / kQ4Step; }
inline int64_t q4_quads(int64_t k) { return (q4_steps(k) + 3) / 4; }
inline int64_t q4_rows16(int64_t rows) { return (rows + 15) / 16 * 16; }

// How a product runs.  bp = 0: the register-fed kernel (few tokens).  bp = 1, 2
// or 4 token panels: k_q4_shared (ap = 8), k cut into `parts`.  Else LDS-fed tiles of ap weight panels x bp token panels, of which the
// first `whole` run over all of k and the others are cut into `parts`.  A gated
// product (`matrices` = 2) takes half of a tile's ap panels from each weight.
struct Q4Route {
  int ap, bp;
  int64_t whole;
  int parts;
};
Q4Route q4_route(int64_t n, int64_t k, int64_t m, int matrices, int64_t cus);
// Workgroups of a route's product (0 for the register-fed kernel).
int64_t q4_groups(const Q4Route& r, int64_t n, int64_t m, int matrices);
// Workspace: a tile's activations as panels, then the parts' sums.
size_t q4_pack_bytes(const Q4Route& r, int64_t k, int64_t m);
size_t q4_part_bytes(const Q4Route& r, int64_t n, int64_t m, int matrices);

hipError_t launch_q4_quantize(const void* a, int dtype, int64_t n, int64_t k, int64_t lda, const hyb_q4& dst,
                              hipStream_t s);
hipError_t launch_q4_dequantize(const hyb_q4& src, int64_t n, int64_t k, void* a, int dtype, int64_t lda,
                                hipStream_t s);
// Y = X W^T, or with `up` act(X W^T) * (X up^T).
hipError_t launch_q4_product(const hyb_q4& w, const hyb_q4* up, int act, int64_t n, int64_t k, const void* x,
                             int x_dtype, int64_t m, int64_t ldx, void* y, int y_dtype, int64_t ldy, char* ws,
                             hipStream_t s);

}  // namespace hyb
