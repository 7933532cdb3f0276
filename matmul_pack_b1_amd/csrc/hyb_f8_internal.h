// Internal interface between the host-side checks of the 8-bit entry points
// (hyb_f8_api.cpp) and their kernels (hyb_f8.hip).  Everything reaching a
// launcher has been validated.
#pragma once

#include "../../include/hyb_f8.h"
#include "hyb_internal.h"

namespace hyb {

// Columns of one step, and its bytes per 16-row panel.
constexpr int64_t kF8Step = 128;
constexpr int64_t kPanelStep = 2048;
// Largest k: a panel's byte offsets within a 16-panel tile stay below 2^31.
constexpr int64_t kF8MaxK = int64_t(1) << 22;
// Launch limits: 512 threads per panel of w, or per tile, stay below 2^32 in
// one grid dimension.
constexpr int64_t kF8MaxRows = (int64_t(1) << 27) - 16;
constexpr int64_t kF8MaxPanelPairs = int64_t(1) << 29;
// Largest grid in its second dimension.
constexpr int64_t kF8MaxGridY = 65535;

inline int64_t f8_steps(int64_t k) { return (k + kF8Step - 1) / kF8Step; }
inline int64_t f8_rows16(int64_t rows) { return (rows + 15) / 16 * 16; }

// How a product runs.
struct F8Route {
  int ap, bp;     // panels of w and of x per workgroup
  int waves;      // register-fed: wavefronts cutting k; LDS-fed: 0
  int64_t whole;  // LDS-fed: tiles that run over all of k ...
  int parts;      // ... and the parts each of the others is cut into (1: all run whole)
};
// `wide`: the product of an fp32 output (kF8Wide).
F8Route f8_route(int64_t n, int64_t k, int64_t m, bool wide, int64_t cus);
size_t f8_workspace_bytes(const F8Route& r, int64_t n, int64_t m);
// Bytes that serve both kinds.
size_t f8_workspace_bytes(int64_t n, int64_t k, int64_t m, int64_t cus);

hipError_t launch_f8_quantize(const void* a, int dtype, int64_t rows, int64_t k, int64_t lda, int kind,
                              const hyb_f8& dst, hipStream_t s);
hipError_t launch_f8_dequantize(const hyb_f8& src, int64_t rows, int64_t k, void* a, int dtype, int64_t lda,
                                hipStream_t s);
// Whether the product of activations still in their own type quantises them
// itself (few tokens), and that product.
bool f8_fused(int64_t n, int64_t k, int64_t m, int y_dtype);
hipError_t launch_f8_fused(const hyb_f8& w, int64_t n, int64_t k, const void* x, int x_dtype, int64_t m, int64_t ldx,
                           void* y, int y_dtype, int64_t ldy, hipStream_t s);
// ws NULL runs the route unsplit.  w_pitch: words between w's scale words of
// four steps and the next four (0: its own rows; more for a part of the rows
// of a larger matrix).
hipError_t launch_f8_gemm(const hyb_f8& w, int64_t n, int64_t k, const hyb_f8& x, int64_t m, void* y, int y_dtype,
                          int64_t ldy, float* ws, hipStream_t s, int64_t w_pitch = 0);

}  // namespace hyb
