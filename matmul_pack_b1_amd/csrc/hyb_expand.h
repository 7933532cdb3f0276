// Sparse tiles of a packed matrix as dense ones, in panels (hyb_panel.h): the order of
// the stores, which the cross entropy's expanding of a piece of the vocabulary has too, and
// the gated projection's expanding.
#ifndef HYB_EXPAND_H_
#define HYB_EXPAND_H_

#include "hyb_device.h"
#include "hyb_panel.h"
#include "hyb_xent_internal.h"

namespace hyb {
namespace {

// Sixteen columns 16 q.. of a row (q = lane / 16) as the two 16-byte pieces of
// the panel order: half q / 2, units 2 (q % 2) and 2 (q % 2) + 1.
__device__ __forceinline__ void store_row16(char* step, int lane, const uint32_t (&e)[8]) {
  const int q = lane >> 4, r = lane & 15;
  char* p = step + (q >> 1) * 1024 + (2 * (q & 1)) * 256;
  *reinterpret_cast<uint4*>(p + r * 16) = make_uint4(e[0], e[1], e[2], e[3]);
  *reinterpret_cast<uint4*>(p + 256 + r * 16) = make_uint4(e[4], e[5], e[6], e[7]);
}

// The tiles of a packed matrix that a PanelOperand calls spare (all but the dense
// ones with a slot), each at its place in tile order in `out`.
struct Expand {
  const char* val;
  const char* meta;
  const int32_t* tidx;
  int32_t n_dense, n_sparse;
  int b1, b2, meta_kind;
  int32_t tiles_k, steps;
  char* out;
};

// Steps s0 .. s0 + 3 of a panel by a wavefront, whose loads are under way at once: two
// weights of 17408 x 5120, 60% of the tiles sparse, 56 us (one step a wavefront, 79).
__device__ __forceinline__ void expand4(const Expand& w, int64_t panel, int32_t s0, int lane) {
  const int64_t r0 = panel * 16, tn = r0 / w.b1;
  const int rs = int(r0 - tn * w.b1) / 16, spt = w.b2 / 64;
  int32_t ti[4];
  uint4 val[4];
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ti[i] = s0 + i < w.steps ? w.tidx[tn * w.tiles_k + (s0 + i) / spt] : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (a tile that is not sparse, or has no slot: an empty resource, zeros)
    const int64_t slot = ~ti[i];
    const bool in = ti[i] < 0 && slot < w.n_sparse && s0 + i < w.steps;
    const int c = (s0 + i) % spt;
    const int64_t at = (in ? slot * w.b1 * w.b2 : 0) + rs * 16 * w.b2;
    const __amdgpu_buffer_rsrc_t vr = make_rsrc(w.val + at + c * 1024, in ? 1024 : 0);
    const __amdgpu_buffer_rsrc_t mr = make_rsrc(w.meta + at / 8, in ? 2 * w.b2 : 0);
    val[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(vr, lane * 16, 0, 0));
    code[i] = __builtin_amdgcn_raw_buffer_load_b16(mr, (lane * spt + c) * 2, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t s = s0 + i;
    if (s >= w.steps || (ti[i] >= 0 && ti[i] < w.n_dense)) continue;
    const bool in = ti[i] < 0 && ~ti[i] < w.n_sparse;
    const uint32_t v[4] = {val[i].x, val[i].y, val[i].z, val[i].w};
    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in && w.meta_kind == HYB_META_MASK8) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[4 * g + j] = __builtin_amdgcn_perm(v[2 * g + 1], v[2 * g], expand8_selector((code[i] >> (8 * g)) & 0xFFu, j));
    } else if (in) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t i0, i1;
        nibble_positions((code[i] >> (4 * g)) & 0xFu, w.meta_kind, i0, i1);
        x[2 * g] = __builtin_amdgcn_perm(0u, v[g], scatter_selector(0, i0, i1));
        x[2 * g + 1] = __builtin_amdgcn_perm(0u, v[g], scatter_selector(2, i0, i1));
      }
    }
    store_row16(w.out + (tn * w.tiles_k + s / spt) * w.b1 * w.b2 * 2 + int64_t(rs) * 32 * w.b2 + s % spt * kPanelStep,
                lane, x);
  }
}

}  // namespace
}  // namespace hyb
#endif  // HYB_EXPAND_H_
