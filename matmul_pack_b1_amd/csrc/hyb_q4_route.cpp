// Host routing of the 4-bit product.
#include "hyb_q4_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens that the register-fed kernel takes.
constexpr int64_t kRowsTokens = 16;

}  // namespace

Q4Route q4_route(int64_t n, int64_t k, int64_t m, int matrices, int64_t cus) {
  if (m <= kRowsTokens) return Q4Route{0, 1, 1};
  Q4Route r{};
  if (m <= 32) r = Q4Route{8, 2, 1};
  else if (m <= 64) r = Q4Route{8, 4, 1};
  else if (m <= 128) r = Q4Route{16, 8, 1};
  else r = Q4Route{16, 16, 1};
  if (r.ap == 16 && r.bp == 16 && q4_tiles(r, n, m, matrices) * 2 <= cus) r.bp = 8;
  const int64_t tiles = q4_tiles(r, n, m, matrices), slots = r.ap == 8 ? 3 * cus : cus;
  const int64_t quads = q4_quads(k);
  double least = 1e300;
  for (int64_t parts = 1; parts <= quads && parts <= 32; ++parts) {
    const double cost = double(up(tiles * parts, slots)) * double(up(quads, parts)) + (parts > 1 ? 0.3 * double(parts) : 0.0);
    if (cost < least) {
      least = cost;
      r.parts = int(parts);
    }
    if (tiles * parts >= 2 * slots) break;
  }
  return r;
}

int64_t q4_tiles(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  return r.ap == 0 ? 1 : up(n, 16 * r.ap / matrices) * up(m, 16 * r.bp);
}

size_t q4_pack_bytes(const Q4Route& r, int64_t k, int64_t m) {
  return r.ap == 0 ? 0 : size_t(up(m, 16)) * size_t(up(k, 64)) * 2048;
}

size_t q4_part_bytes(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  return r.ap == 0 || r.parts <= 1 ? 0 : size_t(q4_tiles(r, n, m, matrices)) * r.parts * r.ap * r.bp * 1024;
}

}  // namespace hyb
