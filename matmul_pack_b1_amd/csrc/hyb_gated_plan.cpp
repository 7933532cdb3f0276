// Host planning of the gated projection over packed weights: routes, tile
// shapes and the workspace.
#include "hyb_gated_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

}  // namespace

GatedPlan gated_plan(const hyb_gated_pair& w, int64_t m, int what, int64_t cus) {
  GatedPlan p{};
  const hyb_layout& L = *w.gate_layout;
  p.n = L.n;
  p.k = L.k;
  p.m = m;
  p.m16 = up(m, 16);
  p.m64 = up(m, 64);
  p.parts = 1;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += size_t(up(bytes, 256));
    return here;
  };
  const bool dx = what & HYB_GATED_DX, dw = what & HYB_GATED_DW;
  const hyb_layout* both[2] = {w.gate_layout, w.up_layout};
  if (!dx && !dw) {
    p.decode = m <= kGemvCrossoverM || (m <= kMaxGemvM && gemv_preferred(L, int(m)));
    p.rows = p.decode || m <= 64;
    p.bp = up(p.n, 128) / 128 * (up(m, 256) / 256) * 2 <= cus || m <= 128 ? 8 : 16;
    if (p.rows) {
      p.gu = take(2 * m * p.n * 4);
      if (!p.decode) {
        for (const hyb_layout* l : both) {
          const size_t need = split_workspace_bytes(gemm_route_device(*l, int(m)));
          if (need > p.split_bytes) p.split_bytes = need;
        }
        p.split = take(int64_t(p.split_bytes));
      }
      p.total = at;
      return p;
    }
  }
  if (!dx && !dw) {
    p.x = take(p.m16 * p.k * 2);
  } else {
    if (dw) p.x = take(p.m16 * p.k * 2);
    p.misc = take(256);
    for (int i = 0; i < 2; ++i) p.g[i] = take(p.m16 * p.n * 2);
    p.bp = m <= 64 ? 4 : m <= 128 ? 8 : 16;
  }
  if (!dw || dx)
    for (int i = 0; i < 2; ++i)
      if (both[i]->n_sparse > 0) p.w[i] = take(p.n * p.k * 2);
  if (dx) {
    const int64_t tiles = up(p.k, 256) / 256 * (up(p.m16, 16 * p.bp) / (16 * p.bp));
    const int64_t slots = p.bp == 4 ? 2 * cus : cus, quads = up(p.n, 256) / 256;
    double least = 1e300;
    for (int parts = 1; parts <= 32 && parts <= quads; ++parts) {
      const double cost = double(up(tiles * parts, slots) / slots) / parts * (1.0 + 0.01 * parts);
      if (cost < least) {
        least = cost;
        p.parts = parts;
      }
    }
    if (p.parts > 1) p.dx = take(int64_t(p.parts) * m * p.k * 4);
  }
  p.total = at;
  return p;
}

}  // namespace hyb
