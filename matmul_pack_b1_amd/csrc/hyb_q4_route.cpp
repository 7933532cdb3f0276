// Host routing of the 4-bit product: the kernel, tile and cuts of k with the
// smallest estimated time.
//
// The estimates' constants are microseconds on an MI355X, fitted to n x k =
// 17408x5120, 14336x4096, 8192x28672, 4096x4096, 5003x1504, 1024x8192 and 500x700
// at 1 to 2048 tokens with up to forty of the choices each, and (gated) 17408x5120,
// 4096x4096 and 2816x1024 (the pick is then 3% above the fastest of them in the
// mean).  Both sides of the choices, at 77 tokens: 5003x1504 k_q4_shared 8.5, tiles
// 18.7; 8192x28672 91 and 66 (k in 8 parts).
#include "hyb_q4_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens that the register-fed kernel takes (17408x5120 at 1 / 2 / 4 tokens 12.1 /
// 13.1 / 15.7 us, k_q4_shared 16.2 / 16.3 / 16.3; at 8 the latter 16.7).
constexpr int64_t kRowsTokens = 4;

int64_t tiles_of(const Q4Route& r, int64_t n, int64_t m, int matrices) {
  return (r.ap == 8 ? up(n, 128) : up(n, 16 * r.ap / matrices)) * up(m, 16 * r.bp);
}

}  // namespace

Q4Route q4_route(int64_t n, int64_t k, int64_t m, int matrices, int64_t cus) {
  if (m <= kRowsTokens) return Q4Route{0, 0, 0, 1};
  const int64_t quads = q4_quads(k);
  Q4Route best{};
  double least = 1e300;
  auto offer = [&](const Q4Route& r, double us) {
    if (us < least) {
      least = us;
      best = r;
    }
  };
  // k_q4_shared: a workgroup's 512 columns take a compute unit `one` us alone on
  // it, `more` us of several, `again` where other token blocks have brought the
  // weights into the caches.  (Rows of fewer than eight columns: tiles.)
  struct Shared {
    int bp;
    double one, more, again;
  };
  for (const Shared& c : {Shared{1, 1.95, 1.71, 1.4}, Shared{2, 2.4, 2.0, 1.9}, Shared{4, 3.4, 3.4, 3.4}}) {
    if (k < 8 || (c.bp > 1 && m <= 8 * c.bp)) continue;
    const int64_t tokens = up(m, 16 * c.bp), blocks = up(n, 128) * tokens;
    if (tokens > 65535) continue;
    for (int64_t parts = 1; parts <= quads && parts <= 16; ++parts) {
      if (parts > 1 && blocks * parts > 8 * cus) break;
      const int64_t deep = up(blocks * parts, cus);
      const double unit = (tokens > 1 && deep > 1 ? c.again : deep > 1 ? c.more : c.one) * (matrices == 2 ? 1.55 : 1.0);
      const double sums = parts > 1 ? 2.6 + double(parts * blocks) * 128 * 16 * c.bp * 8 * matrices / 5.0e6 : 0.0;
      offer(Q4Route{8, c.bp, 0, int(parts)}, 3.4 + double(deep) * double(quads) / double(parts) * unit + sums);
    }
  }
  // LDS-fed tiles: 512 columns of one take a compute unit `one` us, or `more` in
  // several rounds.  Whole rounds of the units run over all of k; the tiles beyond
  // them are cut into parts.
  struct Tile {
    int bp;
    double one, more;
  };
  const double pack = 5.5 + double(m) * double(k) / 1.0e6;
  for (const Tile& c : {Tile{8, 6.6, 5.7}, Tile{16, 11.3, 11.0}}) {
    const Q4Route r{16, c.bp, 0, 1};
    const int64_t tiles = tiles_of(r, n, m, matrices), whole = tiles / cus * cus, rest = tiles - whole;
    const double unit = tiles > cus ? c.more : c.one;
    offer(Q4Route{16, c.bp, tiles, 1}, pack + double(up(tiles, cus) * quads) * unit);
    for (int64_t parts = 2; rest > 0 && parts <= quads && parts <= 32 && rest * parts <= 2 * cus; ++parts) {
      const double sums = 3.0 + double(rest * parts) * 256 * 16 * c.bp * 8 / 7.0e6;
      offer(Q4Route{16, c.bp, whole, int(parts)},
            pack + (double(whole / cus * quads) + double(up(rest * parts, cus)) * double(quads) / double(parts)) * unit + sums);
    }
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
