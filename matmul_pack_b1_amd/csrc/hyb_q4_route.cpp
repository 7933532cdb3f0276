// Host routing of the 4-bit product.
#include "hyb_q4_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens that the register-fed kernel takes, and k_q4_shared.
constexpr int64_t kRowsTokens = 4;
constexpr int64_t kSharedTokens = 64;

int64_t tiles_of(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  return (r.ap == 8 ? up(n, 128) : up(n, 16 * r.ap / matrices)) * up(m, 16 * r.bp);
}

}  // namespace

Q4Route q4_route(int64_t n, int64_t k, int64_t m, int matrices, int64_t cus) {
  if (m <= kRowsTokens) return Q4Route{0, 0, 0, 1};
  const int64_t quads = q4_quads(k);
  if (m <= kSharedTokens) {
    Q4Route r{8, m <= 16 ? 1 : m <= 32 ? 2 : 4, 0, 1};
    const int64_t blocks = up(n, 128), slots = (r.bp == 4 ? 1 : 2) * cus;
    double least = 1e300;
    for (int64_t parts = 1; parts <= quads && parts <= 32; ++parts) {
      const double cost = double(up(blocks * parts, slots)) * (double(up(quads, parts)) + 1.0) + (parts > 1 ? 1.5 : 0.0);
      if (cost < least) {
        least = cost;
        r.parts = int(parts);
      }
    }
    return r;
  }
  Q4Route best{};
  double least = 1e300;
  struct Tile {
    int bp;
    double step;
  };
  for (const Tile& c : {Tile{8, 0.55}, Tile{16, 1.0}}) {
    Q4Route r{16, c.bp, 0, 1};
    const int64_t tiles = tiles_of(r, n, m, matrices), whole = tiles / cus * cus, rest = tiles - whole;
    auto offer = [&](int64_t first, int64_t parts, double cost) {
      if (cost < least) {
        least = cost;
        best = Q4Route{16, c.bp, first, int(parts)};
      }
    };
    offer(tiles, 1, double(up(tiles, cus) * quads) * c.step);
    for (int64_t parts = 2; rest > 0 && parts <= quads && parts <= 32 && rest * parts <= 2 * cus; ++parts)
      offer(whole, parts,
            double(whole / cus * quads + up(rest * parts, cus) * up(quads, parts)) * c.step + 1.0 + 0.002 * double(rest * parts) * c.bp / 16);
  }
  return best;
}

int64_t q4_groups(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  if (r.bp == 0) return 0;
  const int64_t tiles = tiles_of(r, n, m, matrices);
  return r.whole + (tiles - r.whole) * r.parts;
}

size_t q4_pack_bytes(const Q4Route& r, int64_t k, int64_t m) {
  return r.ap != 16 ? 0 : size_t(up(m, 16)) * size_t(up(k, 64)) * 2048;
}

size_t q4_part_bytes(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  if (r.bp == 0 || r.parts <= 1) return 0;
  const size_t each = size_t(r.ap) * r.bp * 1024 * (r.ap == 8 ? matrices : 1);
  return size_t(q4_groups(r, n, m, matrices) - r.whole) * each;
}

}  // namespace hyb
