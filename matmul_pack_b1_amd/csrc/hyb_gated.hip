// Kernels of the gated projection over packed weights (include/hyb_gated.h).
//
// Forward: a tile holds the same rows of the gate and the up projection, so
// that a wavefront ends with G and U of the same outputs in its registers and H
// leaves without a round trip.  Few tokens take the decode or matrix-core
// products of hyb.h into the workspace.  Backward: dG and dU as 16-bit panels
// from one pass over G, U and dH, then dX = dG W_g' + dU W_u' in one product
// over both (W' transposed on its way out of LDS) and dW = dG^T X, dU^T X.
#include <type_traits>

#include "hyb_act.h"
#include "hyb_expand.h"
#include "hyb_gated_internal.h"
#include "hyb_panel.h"
#include "hyb_q4_internal.h"
#include "hyb_stream.h"

namespace hyb {
namespace {

#define HYB_TRY(call)                      \
  do {                                     \
    const hipError_t e_ = (call);          \
    if (e_ != hipSuccess) return e_;       \
  } while (0)

struct GatedOut {
  uint16_t* h;
  float *g, *u;  // NULL: not kept
  int64_t ldh, ldg, ldu;
  int32_t m, n;
  int act;
  // tiles that run over all of k, and the parts each of the others is cut into,
  // whose sums are left in `ws`
  f32x4_t* ws;
  int32_t whole, parts;
};

// Four outputs j.. of a token; fp32 rows may be at any 4-byte aligned address.
template <int DT>
__device__ __forceinline__ void gated_put(const GatedOut& o, int64_t tok, int32_t j, f32x4_t g, f32x4_t u) {
  with_act(o.act, [&](auto act) {
    f32x4_t h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = act_value<decltype(act)::value>(g[e]) * u[e];
    const uint2 r = round16x4<DT>(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<Bytes8*>(o.h + tok * o.ldh + j) = Bytes8{{r.x, r.y}};
  });
}
// (G and U wait for the backward pass: around the caches, 14336x4096, 4096 tokens,
// forward and backward 2530 us instead of 2585, and 2816x1024, 333 tokens 68 either way.)
__device__ __forceinline__ void gated_keep(float* p, f32x4_t v) {
  const u32x4_t b = __builtin_bit_cast(u32x4_t, v);
  stream_store(p, Bytes16{{b[0], b[1], b[2], b[3]}});
}

// H from fp32 G and U, which the products left in memory: four outputs a thread
// (a packed weight's n is a multiple of 64).
template <int DT>
__global__ __launch_bounds__(256) void k_gated_act(GatedOut o) {
  const int64_t tok = blockIdx.y;
  const int32_t j = (int32_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (j >= o.n) return;
  auto load = [&](const float* p) {
    const Bytes16 b = *reinterpret_cast<const Bytes16*>(p);
    return __builtin_bit_cast(f32x4_t, u32x4_t{b.w[0], b.w[1], b.w[2], b.w[3]});
  };
  gated_put<DT>(o, tok, j, load(o.g + tok * o.ldg + j), load(o.u + tok * o.ldu + j));
}

// AP / 2 panels of each weight x BP panels of tokens.  Bound by the matrix units:
// 17408x5120, 2048 tokens 672-696 us in a kernel trace, 1.05-1.09 Pflop/s, of which ten a
// round of tiles are their start, activation and outputs (the whole call takes 652-672 in a
// loop, whose clock is higher); 14336x4096, 4096 tokens with 470 MB of G and U 870-910.
// (A priority above its neighbours' around the matrix instructions: no gain;
// addresses prepared a step earlier 680 against 675 us.)
template <int DT, int AP, int BP, int WA, int WB, int STAGES>
struct GatedTile {
  typedef PanelTile<DT, AP, BP, WA, WB, STAGES, false, false, true, false, true> T;
  static constexpr int kRows = 16 * AP / 2, kOut = T::kA / 2;
};

template <int DT, int AP, int BP, int WA, int WB, int STAGES>
__global__ __launch_bounds__(64 * WA * WB) void k_gated_tile(PanelOperand G, PanelOperand U, PanelOperand X, GatedOut o) {
  typedef GatedTile<DT, AP, BP, WA, WB, STAGES> D;
  typedef typename D::T T;
  constexpr int kOut = D::kOut;
  extern __shared__ __attribute__((aligned(1024))) char gated_smem[];
  const int32_t na = (G.rows16 + D::kRows - 1) / D::kRows, nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  const int32_t id = int32_t(blockIdx.x), rest = id - o.whole;
  const bool cut = rest >= 0;
  int32_t ab, bb;
  panel_block(cut ? o.whole + rest / o.parts : panel_order(id, o.whole), na, nb, ab, bb);
  int32_t s0 = 0, s1 = G.steps;
  if (cut) {
    const int32_t quads = (G.steps + 3) / 4, part = rest % o.parts;  // a part is a whole number of four steps
    s0 = int32_t(int64_t(quads) * part / o.parts) * 4;
    if (part + 1 < o.parts) s1 = int32_t(int64_t(quads) * (part + 1) / o.parts) * 4;
  }
  f32x4_t acc[T::kA][T::kB];
  T::run(G, X, ab * (AP / 2), bb * BP, s0, s1, gated_smem, acc, false, &U);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  if (cut) {
    f32x4_t* out = o.ws + (int64_t(rest) * T::kWaves + wave) * (T::kA * T::kB * 64) + lane;
#pragma unroll
    for (int i = 0; i < T::kA; ++i)
#pragma unroll
      for (int j = 0; j < T::kB; ++j) out[(i * T::kB + j) * 64] = acc[i][j];
    return;
  }
  const int32_t col0 = (ab * (AP / 2) + wa * kOut) * 16, row0 = (bb * BP + wb * T::kB) * 16;
  __syncthreads();  // the tile's LDS stages are free
  if (o.g) {
#pragma unroll
    for (int j = 0; j < T::kB; ++j) {
      const int32_t row = row0 + j * 16 + (lane & 15);
      if (row >= o.m) continue;
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const int32_t col = col0 + i * 16 + (lane >> 4) * 4;
        if (col >= o.n) continue;
        gated_keep(o.g + row * o.ldg + col, acc[i][j]);
        gated_keep(o.u + row * o.ldu + col, acc[i + kOut][j]);
      }
    }
  }
  with_act(o.act, [&](auto act) {
    panel_rows16<kOut, T::kB>(
        gated_smem + wave * (kOut * T::kB * 512), lane, lane & 15,
        [&](int i, int j) {
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = act_value<decltype(act)::value>(acc[i][j][e]) * acc[i + kOut][j][e];
          return round16x4<DT>(v[0], v[1], v[2], v[3]);
        },
        [&](int r, int c, uint4 v) {
          const int32_t row = row0 + r, col = col0 + c;
          if (row < o.m && col < o.n) *reinterpret_cast<Bytes16*>(o.h + row * o.ldh + col) = Bytes16{{v.x, v.y, v.z, v.w}};
        });
  });
}

// Adds the parts of the tiles that were cut, in order: one thread per four
// outputs, in the order of the tile's registers.
template <int DT, int AP, int BP, int WA, int WB, int STAGES>
__global__ __launch_bounds__(256) void k_gated_sum(int32_t na, int32_t nb, GatedOut o) {
  typedef GatedTile<DT, AP, BP, WA, WB, STAGES> D;
  typedef typename D::T T;
  int32_t ab, bb;
  panel_block(o.whole + int32_t(blockIdx.x), na, nb, ab, bb);
  const int lane = threadIdx.x & 63, c = int(blockIdx.y) * 4 + (threadIdx.x >> 6);
  const int wave = c / (D::kOut * T::kB), i = c / T::kB % D::kOut, j = c % T::kB;
  const int32_t col = (ab * (AP / 2) + wave % WA * D::kOut + i) * 16 + (lane >> 4) * 4;
  const int32_t row = (bb * BP + wave / WA * T::kB + j) * 16 + (lane & 15);
  if (row >= o.m || col >= o.n) return;
  f32x4_t v[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const f32x4_t* at = o.ws + (int64_t(blockIdx.x) * o.parts * T::kWaves + wave) * (T::kA * T::kB * 64) +
                        ((i + p * D::kOut) * T::kB + j) * 64 + lane;
    v[p] = at[0];
#pragma unroll 4
    for (int t = 1; t < o.parts; ++t) {
      const f32x4_t u = at[int64_t(t) * T::kWaves * (T::kA * T::kB * 64)];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[p][e] += u[e];
    }
  }
  if (o.g) {
    gated_keep(o.g + row * o.ldg + col, v[0]);
    gated_keep(o.u + row * o.ldu + col, v[1]);
  }
  gated_put<DT>(o, row, col, v[0], v[1]);
}

// ------------------------------------------------------------ the gradients --

struct GatedGrad {
  const float *g, *u;
  const uint16_t* dh;
  int64_t ldg, ldu, lddh;
  int32_t m, n, steps;
  int act;
  char* out[2];   // dG, dU panels: tokens x outputs
  uint32_t* top;  // fp16: bits of the largest finite |dG|, |dU|, then each group's
  int32_t groups;
};

// Four outputs' G, U (fp32) and dH, as loaded from any element-aligned address,
// and their dG and dU.
template <int DT>
struct Gated4 {
  Bytes16 g, u;
  Bytes8 dh;
  __device__ __forceinline__ Gated4() {}
  __device__ __forceinline__ Gated4(const float* gp, const float* up, const uint16_t* dp)
      : g(*reinterpret_cast<const Bytes16*>(gp)),
        u(*reinterpret_cast<const Bytes16*>(up)),
        dh(*reinterpret_cast<const Bytes8*>(dp)) {}
  template <int ACT>
  __device__ __forceinline__ void gradients(float* dg, float* du) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a;
      const float slope = act_slope<ACT>(__builtin_bit_cast(float, g.w[e]), &a);
      const float d = widen16<DT>((dh.w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
      dg[e] = d * __builtin_bit_cast(float, u.w[e]) * slope;
      du[e] = d * a;
    }
  }
};

// The power of two that brings a magnitude of these bits to [2^14, 2^15) (1 for
// zero), and its reciprocal: below fp16's 65504, and 2^-28 of it and above are normal
// numbers (from 2^-14 on).  (A largest below 2^-112, whose factor would not be a
// number, gives zeros in fp16 whatever it is multiplied by.)
__device__ __forceinline__ float gated_lift(uint32_t top, float* back) {
  int e = top == 0 ? 0 : 14 + 127 - int(top >> 23);
  e = e > 126 ? 126 : e;  // (-113 at least, for a finite one)
  *back = __builtin_bit_cast(float, uint32_t(127 - e) << 23);
  return __builtin_bit_cast(float, uint32_t(127 + e) << 23);
}

// Largest finite |dG|, |dU| (fp16) of each workgroup's outputs: one pass over G, U
// and dH more, 5.7 us at 2816x1024 and 333 tokens, 122 at 14336x4096 and 4096 (587 MB, 4.8
// TB/s; forward and backward 2702 us, in bf16 2510).  (Maxima: their order does not
// matter.)
constexpr int kTopGroups = 512;
template <int DT>
__global__ __launch_bounds__(256) void k_gated_top(GatedGrad o) {
  __shared__ uint32_t tops[4];
  uint32_t best = 0;
  const int32_t per = o.n / 4;  // a packed weight's n is a multiple of 64
  const int64_t all = int64_t(o.m) * per;
#pragma unroll 2
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int64_t t = i / per, c = i - t * per;
    float dg[4], du[4];
    const Gated4<DT> in(o.g + t * o.ldg + c * 4, o.u + t * o.ldu + c * 4, o.dh + t * o.lddh + c * 4);
    with_act(o.act, [&](auto act) { in.template gradients<decltype(act)::value>(dg, du); });
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = __builtin_bit_cast(uint32_t, dg[e]) & 0x7FFFFFFFu;
      const uint32_t b = __builtin_bit_cast(uint32_t, du[e]) & 0x7FFFFFFFu;
      if (a < 0x7F800000u && a > best) best = a;
      if (b < 0x7F800000u && b > best) best = b;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t v = __shfl_xor(best, d);
    best = v > best ? v : best;
  }
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 4; ++i) best = tops[i] > best ? tops[i] : best;
    o.top[1 + blockIdx.x] = best;
  }
}

// dG and dU as panels, in the column order in which a lane of the dX product
// holds the rows of a W' that is read transposed (hyb_panel.h): unit u of a half
// has columns 16 (u / 2) + 4 (u % 2) + {0..3, 8..11}.  Rows behind m are zero.
// Bound by memory: 4096 x 14336, 587 MB read and 235 written, 182 us alone (4.5 TB/s;
// in k_gated_prepare the panels of some tokens first, 228 us in all instead of 206).
template <int DT>
__device__ __forceinline__ void gated_grad(const GatedGrad& o, int64_t panel, int32_t quad) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t s = quad * 4 + wave;
  float lift = 1.f;
  if constexpr (DT == HYB_F16) {
    // the largest of the groups' (every workgroup takes it itself)
    __shared__ uint32_t tops[4];
    uint32_t top = 0;
    for (int32_t i = threadIdx.x; i < o.groups; i += 256) top = o.top[1 + i] > top ? o.top[1 + i] : top;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t v = __shfl_xor(top, d);
      top = v > top ? v : top;
    }
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    for (int i = 0; i < 4; ++i) top = tops[i] > top ? tops[i] : top;
    if (panel == 0 && quad == 0 && threadIdx.x == 0) *o.top = top;
    float back;
    lift = gated_lift(top, &back);
  }
  if (s >= o.steps) return;
  const int64_t tok = panel * 16 + (lane & 15);
  // (a lane behind the last token loads the last one's, so that no load branches
  // and all are under way at once)
  const int u4 = lane >> 4;
  const int64_t row = tok < o.m ? tok : o.m - 1, col = s * 64 + 16 * (u4 >> 1) + 4 * (u4 & 1);
  const float *g = o.g + row * o.ldg + col, *u = o.u + row * o.ldu + col;
  const uint16_t* dh = o.dh + row * o.lddh + col;
  Gated4<DT> in[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int p = 0; p < 2; ++p) in[h][p] = Gated4<DT>(g + h * 32 + p * 8, u + h * 32 + p * 8, dh + h * 32 + p * 8);
  const bool live = tok < o.m;
  with_act(o.act, [&](auto act) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float dg[8], du[8];
      in[h][0].template gradients<decltype(act)::value>(dg, du);
      in[h][1].template gradients<decltype(act)::value>(dg + 4, du + 4);
      const int64_t at = (panel * o.steps + s) * kPanelStep + h * 1024 + lane * 16;
      auto put = [&](char* to, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(to + at) =
            live ? make_uint4(round16x2<DT>(v[0] * lift, v[1] * lift), round16x2<DT>(v[2] * lift, v[3] * lift),
                              round16x2<DT>(v[4] * lift, v[5] * lift), round16x2<DT>(v[6] * lift, v[7] * lift))
                 : make_uint4(0, 0, 0, 0);
      };
      put(o.out[0], dg);
      put(o.out[1], du);
    }
  });
}

// What the products read, in one launch (its parts wait for nothing of each
// other, and small calls are the depth of their launches): workgroups of dG and dU
// (backward only), of each weight's sparse tiles, and of x as panels.  2816x1024, 333
// tokens, forward and backward 68 us, with a launch each 76; 14336x4096, 4096 tokens,
// backward 206 us, with a launch each 227 (182, 5.5 TB/s, with G and U past the caches).
struct GatedPrepare {
  GatedGrad grad;
  Expand w[2];
  const uint16_t* x;
  int64_t ldx;
  char* xt;
  int32_t m, k, steps;         // x: tokens, columns, steps of 64
  int32_t grads, weights[2], xs;  // workgroups of each part
};

// x (16-byte aligned rows, k a multiple of 64): a wavefront per panel and four
// steps, whose eight loads are under way at once; rows behind m are zero.
__device__ __forceinline__ void gated_pack_x(const GatedPrepare& o, int64_t panel, int32_t s, int lane) {
  const int64_t row = panel * 16 + (lane & 15);
  const int32_t c0 = s * 64 + (lane >> 4) * 8;
  uint4 u[8];
#pragma unroll
  for (int h = 0; h < 8; ++h)
    u[h] = row < o.m && c0 + h * 32 < o.k ? *reinterpret_cast<const uint4*>(o.x + row * o.ldx + c0 + h * 32)
                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int h = 0; h < 8; ++h)
    if (s + h / 2 < o.steps)
      *reinterpret_cast<uint4*>(o.xt + (panel * o.steps + s) * kPanelStep + h * 1024 + lane * 16) = u[h];
}

template <int DT, bool GRAD>
__global__ __launch_bounds__(256) void k_gated_prepare(GatedPrepare o, int32_t first) {
  int32_t id = first + int32_t(blockIdx.x);
  if constexpr (GRAD) {
    if (id < o.grads) {
      const int32_t quads = (o.grad.steps + 3) / 4;
      return gated_grad<DT>(o.grad, id / quads, id % quads);
    }
    id -= o.grads;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t across = (o.steps + 15) / 16;
  const bool x = id >= o.weights[0] + o.weights[1], second = !x && id >= o.weights[0];
  if (x || second) id -= o.weights[0];
  if (x) id -= o.weights[1];
  const int64_t panel = id / across;
  const int32_t s = (id % across * 4 + wave) * 4;
  if (s >= o.steps) return;
  if (x)
    gated_pack_x(o, panel, s, lane);
  else
    expand4(second ? o.w[1] : o.w[0], panel, s, lane);
}

struct GatedDx {
  float* acc;  // parts: [part][row][k] fp32
  uint16_t* dx;
  int64_t lddx;
  int32_t m, k;
  const uint32_t* top;
};

// dX[token, column] = sum over the outputs of dG W_g' + dU W_u' (A = W' read
// transposed, B = the panels).  A part takes the same steps of both.  14336x4096,
// 4096 tokens 760 us, 1.27 Pflop/s (a library's product 4096 x 14336 x 4096: 1.29).
template <int DT, int AP, int BP, int WA, int WB, int STAGES>
__device__ __forceinline__ void gated_dx(const PanelOperand& G, const PanelOperand& U, const PanelOperand& DG,
                                         const PanelOperand& DU, int32_t steps, int parts, const GatedDx& o, int32_t id,
                                         int32_t part, char* gated_smem) {
  typedef PanelTile<DT, AP, BP, WA, WB, STAGES, true, false, true> T;
  const int32_t na = (G.steps * 4 + AP - 1) / AP, nb = (DG.rows16 / 16 + BP - 1) / BP;
  int32_t ab, bb;
  panel_block(panel_order(id, na * nb), na, nb, ab, bb);
  const int32_t quads = (steps + 3) / 4;  // a part is a whole number of four steps
  const int32_t s0 = int32_t(int64_t(quads) * part / parts) * 4;
  const int32_t s1 = part + 1 == parts ? steps : int32_t(int64_t(quads) * (part + 1) / parts) * 4;
  f32x4_t acc[T::kA][T::kB];
  T::run(G, DG, ab * AP, bb * BP, s0, s1, gated_smem, acc);
  __syncthreads();  // the first product's last stages are free
  T::run(U, DU, ab * AP, bb * BP, s0, s1, gated_smem, acc, true);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave % WA, wb = wave / WA;
  const int32_t row0 = (bb * BP + wb * T::kB) * 16, col0 = (ab * AP + wa * T::kA) * 16;
  if (parts > 1) {
#pragma unroll
    for (int j = 0; j < T::kB; ++j) {
      const int32_t row = row0 + j * 16 + (lane & 15);
      if (row >= o.m) continue;
#pragma unroll
      for (int i = 0; i < T::kA; ++i) {
        const int32_t col = col0 + i * 16 + (lane >> 4) * 4;
        if (col < o.k) *reinterpret_cast<f32x4_t*>(o.acc + (int64_t(part) * o.m + row) * o.k + col) = acc[i][j];
      }
    }
    return;
  }
  float back = 1.f;
  if constexpr (DT == HYB_F16) gated_lift(*o.top, &back);
  __syncthreads();  // the tile's LDS stages are free
  panel_rows16<T::kA, T::kB>(
      gated_smem + wave * (T::kA * T::kB * 512), lane, lane & 15,
      [&](int i, int j) {
        const f32x4_t v = acc[i][j];
        return round16x4<DT>(v[0] * back, v[1] * back, v[2] * back, v[3] * back);
      },
      [&](int r, int c, uint4 u) {
        const int32_t row = row0 + r, col = col0 + c;  // a packed weight's k is a multiple of 64
        if (row < o.m && col < o.k)
          *reinterpret_cast<Bytes16*>(o.dx + row * o.lddx + col) = Bytes16{{u.x, u.y, u.z, u.w}};
      });
}

template <int DT, int AP, int BP, int WA, int WB, int STAGES>
__global__ __launch_bounds__(64 * WA * WB) void k_gated_dx(PanelOperand G, PanelOperand U, PanelOperand DG,
                                                           PanelOperand DU, int32_t steps, int parts, GatedDx o) {
  extern __shared__ __attribute__((aligned(1024))) char gated_smem[];
  gated_dx<DT, AP, BP, WA, WB, STAGES>(G, U, DG, DU, steps, parts, o, int32_t(blockIdx.x), int32_t(blockIdx.y),
                                       gated_smem);
}

// dX = the sum of the parts, in order, rounded once.
template <int DT>
__global__ __launch_bounds__(256) void k_gated_dx_sum(int parts, GatedDx o) {
  const int64_t tok = blockIdx.x;
  const int32_t col = (int32_t(blockIdx.y) * 256 + threadIdx.x) * 4;
  if (col >= o.k) return;
  float back = 1.f;
  if constexpr (DT == HYB_F16) gated_lift(*o.top, &back);
  f32x4_t v = *reinterpret_cast<const f32x4_t*>(o.acc + tok * o.k + col);
#pragma unroll 8
  for (int p = 1; p < parts; ++p) {
    const f32x4_t u = *reinterpret_cast<const f32x4_t*>(o.acc + (int64_t(p) * o.m + tok) * o.k + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += u[e];
  }
  const uint2 r = round16x4<DT>(v[0] * back, v[1] * back, v[2] * back, v[3] * back);
  *reinterpret_cast<Bytes8*>(o.dx + tok * o.lddx + col) = Bytes8{{r.x, r.y}};
}

struct GatedDw {
  uint16_t* dw[2];
  int64_t ld[2];
  int32_t n, k;
  const uint32_t* top;
};

// dW[output, column] = sum over the tokens of dG^T X (both read transposed); the
// grid's second dimension is the weight.  14336x4096, 4096 tokens 770 us, 1.25 Pflop/s
// (four wavefronts with outputs of 128 x 128 each: 844 against 759; X read where it lies:
// 840 against 775).  Small products take tiles of 128 x 128: 2816x1024, 333 tokens, with
// the gradients' pass 22.6 against 25.3 us; 4096x4096, 1024 tokens 92.5 against 82.6.
template <int DT, int AP, int BP, int WA, int WB>
__device__ __forceinline__ void gated_dw(const PanelOperand& X, const PanelOperand& DG, const PanelOperand& DU,
                                         int32_t steps, const GatedDw& o, int32_t id, bool second, char* gated_smem) {
  typedef PanelTile<DT, AP, BP, WA, WB, 2, true, true> T;
  const int32_t na = (X.steps * 4 + AP - 1) / AP, nb = (DG.steps * 4 + BP - 1) / BP;
  int32_t ab, bb;
  panel_block(panel_order(id, na * nb), na, nb, ab, bb);
  PanelOperand D = DG;
  if (second) D.data = DU.data;
  f32x4_t acc[T::kA][T::kB];
  T::run(X, D, ab * AP, bb * BP, 0, steps, gated_smem, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave % WA, wb = wave / WA;
  float back = 1.f;
  if constexpr (DT == HYB_F16) gated_lift(*o.top, &back);
  // the panels' columns 4..7 and 8..11 of 16 have changed places
  const int row16 = (lane & 3) | (lane & 4) << 1 | (lane & 8) >> 1;
  const int32_t row0 = (bb * BP + wb * T::kB) * 16, col0 = (ab * AP + wa * T::kA) * 16;
  uint16_t* y = second ? o.dw[1] : o.dw[0];
  const int64_t ld = second ? o.ld[1] : o.ld[0];
  __syncthreads();  // the tile's LDS stages are free
  panel_rows16<T::kA, T::kB>(
      gated_smem + wave * (T::kA * T::kB * 512), lane, row16,
      [&](int i, int j) {
        const f32x4_t v = acc[i][j];
        return round16x4<DT>(v[0] * back, v[1] * back, v[2] * back, v[3] * back);
      },
      [&](int r, int c, uint4 u) {
        const int32_t row = row0 + r, col = col0 + c;
        if (row < o.n && col < o.k) *reinterpret_cast<Bytes16*>(y + row * ld + col) = Bytes16{{u.x, u.y, u.z, u.w}};
      });
}

template <int DT, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void k_gated_dw(PanelOperand X, PanelOperand DG, PanelOperand DU,
                                                           int32_t steps, GatedDw o) {
  extern __shared__ __attribute__((aligned(1024))) char gated_smem[];
  gated_dw<DT, AP, BP, WA, WB>(X, DG, DU, steps, o, int32_t(blockIdx.x), blockIdx.y != 0, gated_smem);
}

// Small products, of which neither fills the compute units: dX's tiles and, behind
// them, dW's 128 x 128 ones in one launch (figures at the plan's choice of it).
template <int DT, int BP, int WA, int WB, int STAGES>
__global__ __launch_bounds__(512) void k_gated_both(PanelOperand G, PanelOperand U, PanelOperand DG, PanelOperand DU,
                                                    PanelOperand X, int32_t steps, int parts, GatedDx dx, int32_t tiles,
                                                    int32_t steps_m, GatedDw dw, int32_t tiles_w) {
  extern __shared__ __attribute__((aligned(1024))) char gated_smem[];
  int32_t id = int32_t(blockIdx.x);
  if (id < tiles * parts) {
    gated_dx<DT, 16, BP, WA, WB, STAGES>(G, U, DG, DU, steps, parts, dx, id % tiles, id / tiles, gated_smem);
    return;
  }
  id -= tiles * parts;
  gated_dw<DT, 8, 8, 2, 4>(X, DG, DU, steps_m, dw, id % tiles_w, id >= tiles_w, gated_smem);
}

// dW of an empty batch.
__global__ __launch_bounds__(256) void k_gated_zero(uint16_t* __restrict__ dw, int64_t n, int64_t ld, int32_t k) {
  const int32_t c = int32_t(blockIdx.y) * 256 + threadIdx.x;
  for (int64_t r = blockIdx.x; r < n; r += gridDim.x)
    if (c < k) dw[r * ld + c] = 0;
}

// ----------------------------------------------------------------- launches --

template <typename F>
hipError_t allow_lds(F* fn, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// A packed weight as a tile operand; its sparse tiles lie expanded at `spare`.
PanelOperand weight_operand(const hyb_layout& L, const hyb_packed& P, const char* spare) {
  PanelOperand o{};
  o.rows16 = int32_t(L.n);
  o.steps = int32_t(L.k / 64);
  o.data = static_cast<const char*>(P.dense);
  o.log_b1 = __builtin_ctz(L.b1);
  o.log_b2 = __builtin_ctz(L.b2);
  o.tiles_k = int32_t(L.tiles_k);
  o.n_dense = int32_t(L.n_dense);
  o.plain = L.n;
  o.tidx = P.tidx;
  if (L.n_sparse > 0) {
    o.spare = spare;
    o.spare1 = int32_t(L.tiles_n);
  }
  return o;
}

// Both weights' tiles, and x as panels, as the launch below leaves them.
void weight_pair(const hyb_gated_pair& w, const GatedPlan& p, char* ws, GatedPrepare* o, PanelOperand (&out)[2]) {
  const hyb_layout* L[2] = {w.gate_layout, w.up_layout};
  const hyb_packed* P[2] = {w.gate, w.up};
  for (int i = 0; i < 2; ++i) {
    out[i] = weight_operand(*L[i], *P[i], ws + p.w[i]);
    o->w[i] = Expand{static_cast<const char*>(P[i]->val), static_cast<const char*>(P[i]->meta), P[i]->tidx,
                     int32_t(L[i]->n_dense), int32_t(L[i]->n_sparse), L[i]->b1, L[i]->b2, L[i]->meta,
                     int32_t(L[i]->tiles_k), int32_t(p.k / 64), ws + p.w[i]};
    if (L[i]->n_sparse > 0) o->weights[i] = int32_t(p.n / 16 * ((p.k / 64 + 15) / 16));
  }
}
PanelOperand x_panels(const GatedPlan& p, const void* x, int64_t ldx, char* ws, GatedPrepare* o) {
  o->x = static_cast<const uint16_t*>(x);
  o->ldx = ldx;
  o->xt = ws + p.x;
  o->xs = int32_t(p.m16 / 16 * ((p.k / 64 + 15) / 16));
  return PanelOperand{ws + p.x, int32_t(p.m16), int32_t(p.k / 64), nullptr, 0};
}

template <int DT, bool GRAD>
hipError_t prepare(const GatedPlan& p, GatedPrepare& o, hipStream_t s) {
  o.m = int32_t(p.m);
  o.k = int32_t(p.k);
  o.steps = int32_t(p.k / 64);
  const int32_t all = o.grads + o.weights[0] + o.weights[1] + o.xs, most = 1 << 23;
  for (int32_t first = 0; first < all; first += most) {  // (a launch stays below 2^32 threads)
    const int32_t count = all - first < most ? all - first : most;
    hipLaunchKernelGGL((k_gated_prepare<DT, GRAD>), dim3(unsigned(count)), dim3(256), 0, s, o, first);
    HYB_TRY(hipGetLastError());
  }
  return hipSuccess;
}

template <int DT, int BP, int WA, int WB, int STAGES>
hipError_t run_forward_tile(const PanelOperand (&W)[2], const PanelOperand& X, const GatedOut& o, hipStream_t s) {
  typedef GatedTile<DT, 16, BP, WA, WB, STAGES> D;
  typedef typename D::T T;
  HYB_TRY(allow_lds(&k_gated_tile<DT, 16, BP, WA, WB, STAGES>, T::kLds));
  const int64_t na = (W[0].rows16 + 127) / 128, nb = (X.rows16 + 16 * BP - 1) / (16 * BP), rest = na * nb - o.whole;
  hipLaunchKernelGGL((k_gated_tile<DT, 16, BP, WA, WB, STAGES>), dim3(unsigned(o.whole + rest * o.parts)),
                     dim3(64 * WA * WB), T::kLds, s, W[0], W[1], X, o);
  HYB_TRY(hipGetLastError());
  if (rest == 0) return hipSuccess;
  constexpr int kEach = T::kWaves * D::kOut * T::kB;  // of 64 lanes, a tile
  static_assert(kEach % 4 == 0, "whole workgroups");
  hipLaunchKernelGGL((k_gated_sum<DT, 16, BP, WA, WB, STAGES>), dim3(unsigned(rest), kEach / 4), dim3(256), 0, s,
                     int32_t(na), int32_t(nb), o);
  return hipGetLastError();
}

template <int DT>
hipError_t forward_typed(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int64_t ldx,
                         const GatedForward& f, char* ws, hipStream_t s) {
  GatedOut o{};
  o.h = static_cast<uint16_t*>(f.h);
  o.g = f.g;
  o.u = f.u;
  o.ldh = f.ldh;
  o.ldg = f.ldg;
  o.ldu = f.ldu;
  o.m = int32_t(p.m);
  o.n = int32_t(p.n);
  o.act = act;
  if (p.decode)
    return launch_gemv_gated(*w.gate_layout, *w.gate, *w.up_layout, *w.up, act, x, int(p.m), ldx, f.h, f.ldh, f.g, f.ldg,
                             f.u, f.ldu, s);
  if (p.rows) {
    if (!o.g) {  // not kept: in the workspace
      o.g = reinterpret_cast<float*>(ws + p.gu);
      o.u = o.g + p.m * p.n;
      o.ldg = o.ldu = p.n;
    }
    const hyb_layout L[2] = {*w.gate_layout, *w.up_layout};
    const hyb_packed P[2] = {*w.gate, *w.up};
    void* const y[2] = {o.g, o.u};
    const int64_t ldy[2] = {o.ldg, o.ldu};
    if (p.grouped)
      HYB_TRY(launch_gemv_grouped(2, L, P, x, int(p.m), ldx, y, HYB_F32, ldy, s));
    else
      for (int i = 0; i < 2; ++i)
        HYB_TRY(launch_gemm(L[i], P[i], x, int(p.m), ldx, y[i], HYB_F32, ldy[i], s, ws + p.split, p.split_bytes));
    hipLaunchKernelGGL((k_gated_act<DT>), dim3(unsigned((p.n + 1023) / 1024), unsigned(p.m)), dim3(256), 0, s, o);
    return hipGetLastError();
  }
  PanelOperand W[2];
  GatedPrepare first{};
  weight_pair(w, p, ws, &first, W);
  const PanelOperand X = x_panels(p, x, ldx, ws, &first);
  HYB_TRY((prepare<DT, false>(p, first, s)));
  o.ws = reinterpret_cast<f32x4_t*>(ws + p.gu);
  o.whole = int32_t(p.whole);
  o.parts = p.parts;
  if (p.bp == 16) return run_forward_tile<DT, 16, 2, 4, 2>(W, X, o, s);
  if (p.bp == 8) return run_forward_tile<DT, 8, 4, 2, 2>(W, X, o, s);
  return run_forward_tile<DT, 4, 4, 2, 4>(W, X, o, s);
}

template <int DT, int BP, int WA, int WB, int STAGES>
hipError_t run_dx(const PanelOperand (&W)[2], const PanelOperand (&D)[2], int parts, const GatedDx& o, hipStream_t s) {
  typedef PanelTile<DT, 16, BP, WA, WB, STAGES, true, false, true> T;
  HYB_TRY(allow_lds(&k_gated_dx<DT, 16, BP, WA, WB, STAGES>, T::kLds));
  const int64_t na = (W[0].steps * 4 + 15) / 16, nb = (D[0].rows16 / 16 + BP - 1) / BP;
  hipLaunchKernelGGL((k_gated_dx<DT, 16, BP, WA, WB, STAGES>), dim3(unsigned(na * nb), unsigned(parts)), dim3(64 * WA * WB),
                     T::kLds, s, W[0], W[1], D[0], D[1], D[0].steps, parts, o);
  return hipGetLastError();
}

template <int DT, int AP, int BP, int WA, int WB>
hipError_t run_dw(const PanelOperand& X, const PanelOperand (&D)[2], int32_t steps, const GatedDw& o, hipStream_t s) {
  typedef PanelTile<DT, AP, BP, WA, WB, 2, true, true> T;
  HYB_TRY(allow_lds(&k_gated_dw<DT, AP, BP, WA, WB>, T::kLds));
  const int64_t na = (X.steps * 4 + AP - 1) / AP, nb = (D[0].steps * 4 + BP - 1) / BP;
  hipLaunchKernelGGL((k_gated_dw<DT, AP, BP, WA, WB>), dim3(unsigned(na * nb), 2), dim3(64 * WA * WB), T::kLds, s, X, D[0],
                     D[1], steps, o);
  return hipGetLastError();
}

template <int DT, int BP, int WA, int WB, int STAGES>
hipError_t run_both(const PanelOperand (&W)[2], const PanelOperand (&D)[2], const PanelOperand& X, int parts,
                    const GatedDx& dx, int32_t steps_m, const GatedDw& dw, hipStream_t s) {
  typedef PanelTile<DT, 16, BP, WA, WB, STAGES, true, false, true> T;
  typedef PanelTile<DT, 8, 8, 2, 4, 2, true, true> V;
  constexpr int kLds = T::kLds > V::kLds ? T::kLds : V::kLds;
  static_assert(WA * WB == 8, "one size of workgroup");
  HYB_TRY(allow_lds(&k_gated_both<DT, BP, WA, WB, STAGES>, kLds));
  const int64_t tiles = int64_t((W[0].steps * 4 + 15) / 16) * ((D[0].rows16 / 16 + BP - 1) / BP);
  const int64_t tiles_w = int64_t((X.steps * 4 + 7) / 8) * ((D[0].steps * 4 + 7) / 8);
  hipLaunchKernelGGL((k_gated_both<DT, BP, WA, WB, STAGES>), dim3(unsigned(tiles * parts + 2 * tiles_w)), dim3(512), kLds, s,
                     W[0], W[1], D[0], D[1], X, D[0].steps, parts, dx, int32_t(tiles), steps_m, dw, int32_t(tiles_w));
  return hipGetLastError();
}

template <int DT>
hipError_t backward_typed(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int64_t ldx,
                          const GatedBackward& b, char* ws, hipStream_t s) {
  uint32_t* top = reinterpret_cast<uint32_t*>(ws + p.misc);
  GatedPrepare first{};
  GatedGrad& g = first.grad;
  g.g = b.g;
  g.u = b.u;
  g.dh = static_cast<const uint16_t*>(b.dh);
  g.ldg = b.ldg;
  g.ldu = b.ldu;
  g.lddh = b.lddh;
  g.m = int32_t(p.m);
  g.n = int32_t(p.n);
  g.steps = int32_t(p.n / 64);
  g.act = act;
  g.out[0] = ws + p.g[0];
  g.out[1] = ws + p.g[1];
  g.top = top;
  if (DT == HYB_F16) {
    const int64_t want = (p.m * (p.n / 4) + 255) / 256;
    g.groups = int32_t(want < kTopGroups ? want : kTopGroups);
    hipLaunchKernelGGL((k_gated_top<DT>), dim3(unsigned(g.groups)), dim3(256), 0, s, g);
    HYB_TRY(hipGetLastError());
  }
  first.grads = int32_t(p.m16 / 16 * ((g.steps + 3) / 4));
  PanelOperand W[2], X;
  if (b.dx) weight_pair(w, p, ws, &first, W);
  if (b.dw[0]) X = x_panels(p, x, ldx, ws, &first);
  HYB_TRY((prepare<DT, true>(p, first, s)));
  const PanelOperand D[2] = {PanelOperand{ws + p.g[0], int32_t(p.m16), g.steps, nullptr, 0},
                             PanelOperand{ws + p.g[1], int32_t(p.m16), g.steps, nullptr, 0}};
  const GatedDx dx{reinterpret_cast<float*>(ws + p.dx), static_cast<uint16_t*>(b.dx), b.lddx, int32_t(p.m),
                   int32_t(p.k), top};
  const GatedDw dw{{static_cast<uint16_t*>(b.dw[0]), static_cast<uint16_t*>(b.dw[1])}, {b.lddw[0], b.lddw[1]},
                   int32_t(p.n), int32_t(p.k), top};
  const int32_t steps = int32_t(p.m64 / 64);
  const bool both = b.dx && b.dw[0] && p.both;
  if (both) {
    HYB_TRY(p.bp == 16  ? (run_both<DT, 16, 2, 4, 2>(W, D, X, p.parts, dx, steps, dw, s))
            : p.bp == 8 ? (run_both<DT, 8, 4, 2, 2>(W, D, X, p.parts, dx, steps, dw, s))
                        : (run_both<DT, 4, 4, 2, 4>(W, D, X, p.parts, dx, steps, dw, s)));
  } else if (b.dx) {
    HYB_TRY(p.bp == 16  ? (run_dx<DT, 16, 2, 4, 2>(W, D, p.parts, dx, s))
            : p.bp == 8 ? (run_dx<DT, 8, 4, 2, 2>(W, D, p.parts, dx, s))
                        : (run_dx<DT, 4, 4, 2, 4>(W, D, p.parts, dx, s)));
  }
  if (b.dx && p.parts > 1) {
    hipLaunchKernelGGL((k_gated_dx_sum<DT>), dim3(unsigned(p.m), unsigned((p.k + 1023) / 1024)), dim3(256), 0, s, p.parts,
                       dx);
    HYB_TRY(hipGetLastError());
  }
  if (b.dw[0] && !both)
    HYB_TRY(p.small_dw ? (run_dw<DT, 8, 8, 2, 4>(X, D, steps, dw, s)) : (run_dw<DT, 16, 16, 2, 4>(X, D, steps, dw, s)));
  return hipSuccess;
}

}  // namespace

hipError_t launch_gated(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int dtype, int64_t ldx,
                        const GatedForward& out, char* ws, hipStream_t s) {
  return dtype == HYB_BF16 ? forward_typed<HYB_BF16>(w, p, act, x, ldx, out, ws, s)
                           : forward_typed<HYB_F16>(w, p, act, x, ldx, out, ws, s);
}

hipError_t launch_gated_backward(const hyb_gated_pair& w, const GatedPlan& p, int act, const void* x, int dtype,
                                 int64_t ldx, const GatedBackward& b, char* ws, hipStream_t s) {
  if (p.m == 0) {
    for (int i = 0; i < 2; ++i) {
      hipLaunchKernelGGL(k_gated_zero, dim3(unsigned(p.n < 4096 ? p.n : 4096), unsigned((p.k + 255) / 256)), dim3(256), 0,
                         s, static_cast<uint16_t*>(b.dw[i]), p.n, b.lddw[i], int32_t(p.k));
      HYB_TRY(hipGetLastError());
    }
    return hipSuccess;
  }
  return dtype == HYB_BF16 ? backward_typed<HYB_BF16>(w, p, act, x, ldx, b, ws, s)
                           : backward_typed<HYB_F16>(w, p, act, x, ldx, b, ws, s);
}

}  // namespace hyb
