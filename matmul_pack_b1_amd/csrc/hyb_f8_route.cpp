// Host routing of the 8-bit product: the kernel, tile and cuts of k with the
// smallest estimated time.
//
// The estimates' constants are microseconds on an MI355X, fitted to n x k =
// 17408x5120, 5120x17408, 14336x4096, 4096x4096, 8192x28672, 1024x8192,
// 5003x1501 and 500x700 at 1 to 4096 tokens with ten of the choices each (the
// pick is then 0.5% above the fastest of them in the mean).  Both sides of the
// choices, at 77 tokens, bf16 output: 5003x1501 register-fed 8.0, 128x128 tiles
// 12.1, 256x256 32; 17408x5120 60, 21, 58; 5120x17408 63, 55 (23.8 with k in 4
// parts), 167.
#include "hyb_f8_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

F8Route f8_route(int64_t n, int64_t k, int64_t m, bool wide, int64_t cus) {
  const int64_t np = up(n, 16), mp = up(m, 16), steps = f8_steps(k), quads = up(steps, 4);
  F8Route best{};
  double best_us = 1e300;
  auto offer = [&](const F8Route& r, double us) {
    if (us < best_us) {
      best_us = us;
      best = r;
    }
  };
  // w streamed from memory or the last-level cache.
  const double stream = double(n) * double(k) / 9.0e6;
  auto longest = [](double a, double b, double c) {
    const double d = a > b ? a : b;
    return d > c ? d : c;
  };
  // Register-fed, one panel of w by bp of x: a step of a workgroup takes a CU
  // `step` us when there are enough of them, a wavefront's own four steps
  // `quad` us when there are not.
  struct Rows {
    int bp;
    double step, quad;
  };
  for (const Rows& c : {Rows{1, 0.086, 2.0}, Rows{2, 0.125, 3.2}, Rows{4, 0.205, 5.6}}) {
    if (up(mp, c.bp) > kF8MaxGridY) continue;  // its tokens are the grid's second dimension
    const double full = double(np * up(mp, c.bp)) * double(steps) / double(cus) * c.step;
    offer(F8Route{1, c.bp, 8, 0, 1}, 2.4 + longest(full, double(up(quads, 8)) * c.quad, stream));
  }
  // LDS-fed tiles, one per CU at a time: `step` us per step of a tile, and
  // `work` us per step when every CU is busy (the matrix units' own rate).
  // Whole rounds of the CUs first; the tiles left over whole too, or cut into
  // parts, whose fp32 sums are written and read once.
  struct Tile {
    int ap, bp;
    double step, work, wide_step, wide_work;
  };
  for (const Tile& c : {Tile{8, 8, 0.49, 2.4e-3, 1.0, 2.4e-3}, Tile{16, 8, 1.08, 4.7e-3, 1.63, 6.4e-3},
                        Tile{16, 16, 1.78, 7.5e-3, 2.83, 9.4e-3}}) {
    const double step = wide ? c.wide_step : c.step;
    const int64_t tiles = up(np, c.ap) * up(mp, c.bp);
    const int64_t whole = tiles / cus * cus, rest = tiles - whole;
    const double work = double(tiles) * double(steps) * (wide ? c.wide_work : c.work) * 256.0 / double(cus);
    offer(F8Route{c.ap, c.bp, 0, tiles, 1}, 5.0 + longest(double(up(tiles, cus) * steps) * step, work, stream));
    for (int64_t parts = 2; rest > 0 && parts <= quads && parts <= 32 && rest * parts <= 2 * cus; ++parts) {
      const double sums = double(rest * parts) * c.ap * c.bp * 1024 * 2 / 5.3e6;
      const double rounds = double(whole / cus * steps + up(rest * parts, cus) * up(quads, parts) * 4) * step;
      offer(F8Route{c.ap, c.bp, 0, whole, int(parts)}, 8.0 + sums + longest(rounds, work, stream));
    }
  }
  return best;
}

size_t f8_workspace_bytes(const F8Route& r, int64_t n, int64_t m) {
  if (r.parts <= 1) return 0;
  const int64_t tiles = up(n, 16 * r.ap) * up(m, 16 * r.bp);
  return size_t((tiles - r.whole) * r.parts) * r.ap * r.bp * 1024;
}

size_t f8_workspace_bytes(int64_t n, int64_t k, int64_t m, int64_t cus) {
  const size_t a = f8_workspace_bytes(f8_route(n, k, m, false, cus), n, m);
  const size_t b = f8_workspace_bytes(f8_route(n, k, m, true, cus), n, m);
  return a > b ? a : b;
}

}  // namespace hyb
