// Host planning of the cross entropy: pieces of the vocabulary, tile shapes
// and the workspace.
#include "hyb_xent_internal.h"

namespace hyb {

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

}  // namespace

XentPlan xent_plan(const hyb_head& head, int64_t m, int what, int64_t cus) {
  XentPlan p{};
  p.f8 = head.f8 != nullptr;
  p.n = p.f8 ? head.n : head.layout->n;
  p.k = p.f8 ? head.k : head.layout->k;
  p.m = m;
  p.m16 = up(m, 16);
  p.m64 = up(m, 64);
  p.steps = p.f8 ? f8_steps(p.k) : p.k / 64;
  p.ksteps16 = p.f8 ? 2 * p.steps : p.steps;
  const bool dx = what & HYB_XENT_DX, dw = what & HYB_XENT_DW;
  // The loss alone: for few tokens the logits of a piece go through the
  // library's product and the workspace (33 MB at 64 tokens x 128256), which
  // reads the head once as it lies.  A packed head with sparse tiles would have
  // to be expanded for the tiles below, which costs more than the logits'
  // round trip up to about 512 tokens (128256 x 4096, 60% of the tiles sparse,
  // bf16, 100 / 256 / 512 / 1024 tokens: 345 / 386 / 610 / 1127 us through the
  // product, 669 / 674 / 707 / 1144 through the tiles; 10% sparse, 512 tokens:
  // 664 and 609).
  // So do products of up to an eighth as many tiles of 256 x 256 as there are
  // compute units, for which the library's products have smaller tiles (k is not
  // cut here, even where their route would; loss, dense, k = 4096,
  // entries x tokens: 1024 x 100 27 us, the tiles 61; 4096 x 300, 32 tiles, 37 and
  // 68; 4096 x 1000, 64 tiles, 123 and 70; 8-bit 28 / 59, 47 / 60, 54 / 63; loss and
  // dX of 4096 x 300 104 and 164).
  // Gradients need the expanded tiles anyway; up to 64 tokens their logits go
  // the same way too (16 tokens, 32768 x 4096 of the head: the tile of 256 x 64
  // 100 us, the product 40).
  const int64_t few = !dx && !dw && !p.f8 && head.layout->n_sparse > 0 ? 512 : 64;
  p.rows = m <= few || up(p.n, 256) / 256 * (up(m, 256) / 256) * 8 <= cus;
  // Pieces of 32768 entries (at 4096 tokens 2048 tiles of 256 x 256, eight rounds
  // of 256 compute units), fewer where their 16-bit dz would pass 256 MiB.  Few
  // tokens take more, up to 64 MiB of dz, which fills the units and saves
  // launches (loss and dX, dense 128256 x 4096, 16 / 64 / 100 tokens: pieces of
  // 32768 606 / 725 / 883 us, whole 577 / 666 / 676); over sparse tiles as far as
  // the expanded copy of a piece stays within 512 MiB.
  const int64_t dz = 2 * (p.m64 > 0 ? p.m64 : 64);
  p.piece = (int64_t(256) << 20) / dz;
  if (p.piece > 32768) {
    int64_t most = (int64_t(64) << 20) / dz;
    if (!p.f8 && head.layout->n_sparse > 0) {
      const int64_t copy = (int64_t(512) << 20) / (2 * p.k);
      most = most < copy ? most : copy;
    }
    if (most > 32768) most = up(p.n, up(p.n, most) / most) / (up(p.n, most) / most);  // even pieces
    p.piece = most > 32768 ? up(most, 256) : 32768;
  }
  p.piece = p.piece < 256 ? 256 : p.piece / 256 * 256;
  if (p.piece > up(p.n, 256)) p.piece = up(p.n, 256);
  // Token panels per tile: fewer where 256 tokens a tile would leave more than
  // half of the compute units without one.
  const int64_t wide = up(p.piece, 256) / 256 * (up(m, 256) / 256);
  p.bp = m <= 64 ? 4 : m <= 128 || 2 * wide <= cus ? 8 : 16;
  if (dx || dw)
    p.at_once = p.piece;
  else if (p.rows)
    p.at_once = m <= 64 ? p.n : 32768;
  else  // a head that is multiplied where it lies is one piece
    p.at_once = p.f8 || head.layout->n_sparse == 0 ? p.n : p.piece;
  if (p.at_once > p.n) p.at_once = p.n;
  p.chunks = p.rows ? up(p.n, 2048) / 2048 : up(p.n, 256) / 256;
  p.parts = 1;
  if (dx) {
    // The dX product has (k / 256) x (m / 256) tiles; its vocabulary is cut
    // into the number of parts that keeps the compute units fullest (rounds of
    // them per part; 1% a part for the sums it writes).  Where two workgroups'
    // LDS fits a unit, one's reads hide behind the other's waits: 16 tokens over
    // an 8-bit 152064 x 5120 head 225 us with one a unit, 149 with two; a packed
    // 64128 x 4096 piece 101 and 89.
    const int64_t tiles = up(p.ksteps16 * 64, 256) / 256 * (up(p.m16, 16 * p.bp) / (16 * p.bp));
    const int64_t slots = p.bp == 4 || (p.bp == 8 && p.f8) ? 2 * cus : cus;
    double least = 1e300;
    const int64_t quads = up(p.piece, 256) / 256;  // of four 64-entry steps, a part at least one
    for (int parts = 1; parts <= 32 && parts <= quads; ++parts) {
      const double cost = double(up(tiles * parts, slots) / slots) / parts * (1.0 + 0.01 * parts);
      if (cost < least) {
        least = cost;
        p.parts = parts;
      }
    }
  }
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += size_t(up(bytes, 256));
    return here;
  };
  const int64_t krows = p.ksteps16 * 64;
  if (p.f8) {
    p.x = take(p.m16 * p.steps * 128);
    p.xs = take((p.steps + 3) / 4 * p.m16 * 4);
  } else if (!p.rows || dw) {
    p.x = take(p.m16 * p.k * 2);
  }
  p.misc = take(256);
  if (!dx && !dw) {
    p.part = take(p.chunks * p.m16 * 8);
    p.zt = take(p.m16 * 4);
  }
  if (p.rows) p.logits = take(m * up(p.at_once, 4) * 4);
  // Expanded tiles: a piece of them over sparse tiles; without any the loss
  // needs none and the gradients one tile row, where the vocabulary may end (loss
  // of 100 tokens over a dense 128256 x 4096 head: 1.4 MB in all, 1052 with a
  // piece).
  if (!p.f8 && (!p.rows || dx)) {
    if (head.layout->n_sparse > 0)
      p.w = take(p.piece * krows * 2);
    else if (dx || dw)
      p.w = take(int64_t(head.layout->b1) * krows * 2);
  }
  if (dx || dw) p.g = take(p.m16 * p.piece * 2);
  if (dx) p.dx = take(int64_t(p.parts) * m * krows * 4);
  p.total = at;
  return p;
}

}  // namespace hyb
