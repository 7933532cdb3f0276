// Host planning of the gated projection over packed weights: routes, tile
// shapes and the workspace.
#include "hyb_gated_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Tiles of 256 rows x 16 bp tokens: microseconds of four 64-column steps on a
// compute unit, and of what comes before and after them.  `sums` and `sum_rate`
// (bytes a microsecond) price the joining of cut tiles; no order of tiles is
// faster than `weight_rate` over the expanded weights.  Fitted to timings of
// every tile and cut that fits at 96 (forward) and 98 (dX) sizes from 1024 x 4096
// to 17408 x 5120, 1 to 4096 tokens: the tile taken is at most 7% slower than
// the best one there, and 0.1% on average (tiles of one size are up to 60% slower).
struct Tile {
  int bp;
  double quad, start;
};
struct Costs {
  Tile tiles[3];
  double sums, sum_rate, weight_rate;
};
constexpr Costs kForward = {{{4, 3.2, 2.6}, {8, 4.8, 5.3}, {16, 6.9, 10.0}}, 4.0, 5.6e6, 4.5e6};
constexpr Costs kInput = {{{4, 3.7, 2.0}, {8, 4.4, 4.8}, {16, 5.3, 8.2}}, 2.2, 9.2e6, 1.0e7};

// Up to this many tokens the forward pass runs the two products of the sparse
// kernels and joins them: 14336 x 4096, 30% sparse, 128 tokens 72 against 89 us,
// 4096 x 4096 37 against 40; at 333 tokens 165 against 136 and 60 against 57.
constexpr int64_t kRowsTokens = 128;

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
    p.decode = m <= kGemvCrossoverM;
    if (p.decode) return p;
    p.rows = m <= kRowsTokens;
    p.grouped = m <= kMaxGemvM && gemv_preferred(L, int(m));
    if (p.rows) {
      p.gu = take(2 * m * p.n * 4);
      if (!p.grouped) {
        for (const hyb_layout* l : both) {
          const size_t need = split_workspace_bytes(gemm_route_device(*l, int(m)));
          if (need > p.split_bytes) p.split_bytes = need;
        }
        p.split = take(int64_t(p.split_bytes));
      }
      p.total = at;
      return p;
    }
    // Whole rounds of the compute units run over all of k; the tiles beyond them
    // are cut into parts.
    const int64_t quads = (p.k / 64 + 3) / 4;
    double least = 1e300;
    const double weights = double(4 * p.n * p.k) / kForward.weight_rate;
    for (const Tile& c : kForward.tiles) {
      const int64_t tiles = up(p.n, 128) / 128 * (up(m, 16 * c.bp) / (16 * c.bp));
      const int64_t whole = tiles / cus * cus, rest = tiles - whole;
      auto offer = [&](int64_t first, int64_t parts, double cost) {
        if (cost < least) {
          least = cost;
          p.bp = c.bp;
          p.whole = first;
          p.parts = int(parts);
        }
      };
      auto longer = [&](double t) { return t > weights ? t : weights; };
      offer(tiles, 1, longer(double(up(tiles, cus) / cus) * (double(quads) * c.quad + c.start)));
      for (int64_t parts = 2; rest > 0 && parts <= quads && parts <= 32 && rest * parts <= 2 * cus; ++parts) {
        const double sums = kForward.sums + double(rest * parts) * 256 * 16 * c.bp * 8 / kForward.sum_rate;
        offer(whole, parts,
              longer(double(whole / cus) * (double(quads) * c.quad + c.start) +
                     double(up(rest * parts, cus) / cus) * (double(quads) / double(parts) * c.quad + c.start)) +
                  sums);
      }
    }
    if (p.parts > 1) {
      const int64_t tiles = up(p.n, 128) / 128 * (up(m, 16 * p.bp) / (16 * p.bp));
      p.gu = take((tiles - p.whole) * p.parts * 16 * p.bp * 1024);
    }
  } else {
    p.misc = take(4 + 512 * 4);  // the largest gradient, and that of each workgroup
    for (int i = 0; i < 2; ++i) p.g[i] = take(p.m16 * p.n * 2);
    // (figures at k_gated_dw)
    p.small_dw = m <= 256 || up(p.n, 256) / 256 * (up(p.k, 256) / 256) * 2 <= cus;
  }
  if (!dx || dw) p.x = take(p.m16 * p.k * 2);
  if (!dw || dx)
    for (int i = 0; i < 2; ++i)
      if (both[i]->n_sparse > 0) p.w[i] = take(p.n * p.k * 2);
  if (dx) {
    // (k / 256) x (m / 16 bp) tiles, whose 2 n outputs are cut into parts
    const int64_t quads = up(p.n, 256) / 256;  // of four steps of each weight
    double least = 1e300;
    const double weights = double(4 * p.n * p.k) / kInput.weight_rate;
    for (const Tile& c : kInput.tiles) {
      const int64_t tiles = up(p.k, 256) / 256 * (up(p.m16, 16 * c.bp) / (16 * c.bp));
      for (int parts = 1; parts <= 32 && parts <= quads; ++parts) {
        if (parts > 1 && tiles * parts > 4 * cus) break;
        const double rounds = double(up(tiles * parts, cus) / cus);
        const double sums =
            parts > 1 ? kInput.sums + double(parts) * double(m) * double(p.k) * 8 / kInput.sum_rate : 0.0;
        const double tile = rounds * (2.0 * double(up(quads, parts) / parts) * c.quad + c.start);
        const double cost = (tile > weights ? tile : weights) + sums;
        if (cost < least) {
          least = cost;
          p.parts = parts;
          p.bp = c.bp;
        }
      }
    }
    // dX's and dW's tiles side by side, one a compute unit (dW's alone: two).  Both
    // gradients in us, a launch each and one: 512x512 333 tokens 28.7, 23.0;
    // 2816x1024 333 tokens 46.4, 39.0, 1024 tokens 65.0, 68.5; 1024x4096 200 tokens
    // 40.3, 38.7, 1024 tokens 65.5, 71.7; 4096x4096 200 tokens 80.7, 87.8.
    const int64_t units = up(p.k, 256) / 256 * (up(p.m16, 16 * p.bp) / (16 * p.bp)) * p.parts;
    const int64_t units_w = 2 * (up(p.n, 128) / 128) * (up(p.k, 128) / 128);
    p.both = dw && p.small_dw && (units + units_w <= cus || (units_w <= 2 * cus && m <= 512));
    if (p.parts > 1) p.dx = take(int64_t(p.parts) * m * p.k * 4);
  }
  p.total = at;
  return p;
}

}  // namespace hyb
