// Kernels of the cross entropy over a vocabulary projection
// (include/hyb_xent.h).
//
// The vocabulary is cut into pieces.  Loss: each 256-entry x 256-token tile of
// Z = W' X^T leaves, per token, the maximum and the sum of exponentials of
// its entries (and the target's logit); a second kernel joins them to lse.
// Gradient: the same tiles, recomputed, become G = softmax - onehot in
// registers and leave as 16-bit panels, from which dX = G W' (summed over
// pieces in fp32) and dW = G^T X follow.  All products run on the panel tiles
// of hyb_panel.h; the operands that the gradients need the other way round
// (W', X and, for dW, G) are transposed on their way out of LDS.
#include <type_traits>

#include "hyb_expand.h"
#include "hyb_panel.h"
#include "hyb_xent_internal.h"

namespace hyb {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// exp(z - x) as exp2(fma(z, log2 e, -hi)) * fix, two instructions an element:
// hi is x log2 e rounded, fix takes its rounding back.  That rounding is half an
// ulp of hi: a sixteenth at |x| = 2^20, but 2^7 from 1.5e9 on and 2^8 from 3e9,
// where one factor can be 0 and the other infinite.  An x beyond kNear is `far`,
// and raw_any takes the difference first (three instructions, fix 1).  Where a
// wavefront has no far x, raw serves it; a near x has the same bits either way.
struct ExpBase {
  static constexpr float kNear = 1048576.f;
  float x, hi, fix;
  bool far;
  __device__ __forceinline__ explicit ExpBase(float at) : x(at) {
    hi = x * kLog2e;
    far = __builtin_fabsf(x) > kNear;
    fix = far ? 1.f : __builtin_amdgcn_exp2f(-__builtin_fmaf(x, kLog2e, -hi));
  }
  __device__ __forceinline__ float raw(float z) const {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -hi));
  }
  __device__ __forceinline__ float raw_any(float z) const { return far ? fast_exp(z - x) : raw(z); }
};

// exp(a - b) for a <= b where both may be -inf (an empty sum): 0.
__device__ __forceinline__ float rescale(float a, float b) { return a == b ? 1.f : fast_exp(a - b); }

// Factor that lifts probabilities into fp16's normal range (bf16 needs none).
template <int DT>
constexpr float g_scale() {
  return DT == HYB_F16 ? 16384.f : 1.f;
}

// ------------------------------------------------------------ operand forms --

// x (m x k, row-major) as panels; rows of ignored tokens and behind m zero.
// Bound by memory (4096 x 4096 17 us, once a call).
__global__ __launch_bounds__(256) void k_xent_pack_x(const uint16_t* __restrict__ x, int64_t ldx, int64_t m,
                                                     int32_t steps, const int64_t* __restrict__ target, int64_t ignore,
                                                     char* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = blockIdx.x;
  const int32_t s = int32_t(blockIdx.y) * 4 + wave;
  if (s >= steps) return;
  const int64_t row = panel * 16 + (lane & 15);
  const bool live = row < m && target[row] != ignore;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live) u = *reinterpret_cast<const uint4*>(x + row * ldx + s * 64 + h * 32 + (lane >> 4) * 8);
    *reinterpret_cast<uint4*>(out + (panel * steps + s) * kPanelStep + h * 1024 + lane * 16) = u;
  }
}

// The tiles of rows v0.. (a multiple of b1) of a packed matrix that are not
// multiplied where they lie, into `out` in tile order (one wavefront per panel
// and step): sparse ones expanded from their values and codes, those of a tile
// row that reaches into the padding with its rows from n_vocab on zero, ones
// without a slot zero.  `plain` as in PanelOperand.  Bound by the writes: 37 us
// for a piece of 32768 x 4096 with 30% of its tiles sparse.
__global__ __launch_bounds__(256) void k_xent_expand(const uint4* __restrict__ dense, const uint4* __restrict__ val,
                                                     const uint16_t* __restrict__ meta,
                                                     const int32_t* __restrict__ tidx, int b1, int b2, int meta_kind,
                                                     int32_t tiles_k, int32_t n_dense, int32_t n_sparse, int64_t v0,
                                                     int64_t n_vocab, int64_t plain, int32_t steps,
                                                     char* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t s = int32_t(blockIdx.y) * 4 + wave;
  if (s >= steps) return;
  const int64_t r0 = v0 + int64_t(blockIdx.x) * 16;  // first row of the panel
  const int64_t tn = r0 / b1;
  const int rs = int(r0 - tn * b1) / 16;              // slab within the tile
  const int spt = b2 / 64, c = s % spt;
  const int32_t ti = tidx[tn * tiles_k + s / spt];
  const bool is_dense = ti >= 0 && ti < n_dense;
  if (is_dense && (tn + 1) * b1 <= plain) return;
  char* dst = out + ((tn - v0 / b1) * tiles_k + s / spt) * b1 * b2 * 2 + int64_t(rs) * 32 * b2 + c * kPanelStep;
  const bool row_ok = r0 + (lane & 15) < n_vocab;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (is_dense) {
    const uint4* src = dense + (int64_t(ti) * b1 * b2 + int64_t(rs) * 16 * b2 + c * 1024) / 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4*>(dst + h * 1024 + lane * 16) = row_ok ? src[h * 64 + lane] : zero;
    return;
  }
  uint32_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (ti < 0 && ~ti < n_sparse && row_ok) {
    const int64_t slot = ~ti;
    const uint4 u = val[(slot * b1 * b2 / 2 + int64_t(rs) * 8 * b2 + c * 512) / 8 + lane];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const uint32_t code = meta[slot * b1 * b2 / 16 + int64_t(rs) * b2 + lane * (b2 / 64) + c];
    if (meta_kind == HYB_META_MASK8) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          e[4 * g + j] = __builtin_amdgcn_perm(w[2 * g + 1], w[2 * g], expand8_selector((code >> (8 * g)) & 0xFFu, j));
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t i0, i1;
        nibble_positions((code >> (4 * g)) & 0xFu, meta_kind, i0, i1);
        e[2 * g] = __builtin_amdgcn_perm(0u, w[g], scatter_selector(0, i0, i1));
        e[2 * g + 1] = __builtin_amdgcn_perm(0u, w[g], scatter_selector(2, i0, i1));
      }
    }
  }
  store_row16(dst, lane, e);
}

// Largest exponent byte of an 8-bit head's scales (rows < n_vocab); *top starts
// at 0.  The fp16 form of its values is divided by 2^(top - 133): at most
// 448 * 64, and exact for blocks whose scale is within 2^21 of the largest
// (smaller ones lose bits of values that are below 2^-30 of the head's
// largest).  bf16 holds every value as it is.
__global__ __launch_bounds__(256) void k_xent_top_scale(const uint32_t* __restrict__ scales, int64_t rows16,
                                                        int64_t n_vocab, int32_t steps, uint32_t* __restrict__ top) {
  const int64_t row = int64_t(blockIdx.x) * 256 + threadIdx.x;
  uint32_t t = 0;
  if (row < n_vocab) {
    const int32_t s0 = int32_t(blockIdx.y) * 4;
    const uint32_t w = scales[int64_t(blockIdx.y) * rows16 + row];
    for (int i = 0; i < 4; ++i)
      if (s0 + i < steps) {
        const uint32_t b = (w >> (8 * i)) & 0xFFu;
        t = b > t ? b : t;
      }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_xor(t, d);
    t = o > t ? o : t;
  }
  if ((threadIdx.x & 63) == 0 && t > 0) atomicMax(top, t);
}

// --------------------------------------------------------------- the logits --

struct XentTile {
  int64_t v0;       // first vocabulary row of the piece
  int64_t n_vocab, ignore;
  const int64_t* target;
  int32_t m, m16;
  // loss
  float2* part;     // [chunk][m16]: maximum, sum of exponentials
  float* zt;        // target's logit
  // gradient
  const float* lse;
  const float* grad;
  const float* gtop;  // power of two >= max |grad|
  char* g;            // panels of diag(grad / gtop) G: tokens x entries of the piece
  int32_t g_steps;
};

// One tile of Z = W' X^T: AP x BP panels (entries x tokens).  GRAD false
// leaves the softmax sums, true G.  Bound by the matrix instructions (and the
// clock they leave): a piece of 32768 x 4096, bf16, 4096 tokens takes 795 us with
// the sums (1.38 PFLOP/s), 834 with G.  What comes after a tile's products
// hides behind no others, a CU's LDS being full with one tile: with comparisons
// for masks and targets at every element and rounding in integers (17
// instructions an element) it was 829 and 939.  The library's plain product of
// that size runs at 1.45 PFLOP/s and leaves the logits to read.
template <int KIND, int DT, bool GRAD, bool TILED, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void k_xent_tile(PanelOperand W, PanelOperand X, XentTile t) {
  typedef PanelTile<KIND, AP, BP, WA, WB, 2, false, false, TILED> T;
  extern __shared__ __attribute__((aligned(1024))) char xent_smem[];
  const int32_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  int32_t ab, bb;
  panel_block(panel_order(int32_t(blockIdx.x), na * nb), na, nb, ab, bb);
  f32x4_t acc[T::kA][T::kB];
  T::run(W, X, ab * AP, bb * BP, 0, W.steps, xent_smem, acc);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  // entry of acc[i][.][e]: vbase + 16 i + e; token of acc[.][j]: tbase + 16 j
  const int64_t vbase = t.v0 + int64_t(ab * AP + wa * T::kA) * 16 + (lane >> 4) * 4;
  const int32_t tbase = (bb * BP + wb * T::kB) * 16 + (lane & 15);
  // entries of this lane's 16 kA that are in the vocabulary, and which of them a
  // target is (-1: none)
  constexpr int kSpan = 16 * T::kA;
  const int32_t live = t.n_vocab - vbase < kSpan ? int32_t(t.n_vocab - vbase) : kSpan;
  const bool edge = __any(live < kSpan);
  auto place = [&](int64_t want) {
    const uint64_t at = uint64_t(want) - uint64_t(vbase);
    return at < uint64_t(kSpan) ? int32_t(at) : -1;
  };
  if constexpr (!GRAD) {
    __syncthreads();  // the tile's LDS stages are free
    float2* sums = reinterpret_cast<float2*>(xent_smem);  // [WA][16 BP]
#pragma unroll
    for (int j = 0; j < T::kB; ++j) {
      const int32_t tok = tbase + 16 * j;
      if (edge) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * i + e >= live) acc[i][j][e] = -__builtin_inff();
      }
      // the target's logit, in the few wavefronts that hold one
      const int32_t at = tok < t.m ? place(t.target[tok]) : -1;
      if (__any(at >= 0)) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at == 16 * i + e) t.zt[tok] = acc[i][j][e];
      }
      // (a maximum passes NaN over; the sum does not)
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < T::kA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __builtin_fmaxf(top, acc[i][j][e]);
#pragma unroll
      for (int d = 16; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
      // an infinite maximum (no entry above -inf, or one of +inf) would give NaN
      const ExpBase base(__builtin_fabsf(top) < __builtin_inff() ? top : 0.f);
      float sum = 0.f;
      if (__any(base.far)) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += base.raw_any(acc[i][j][e]);
      } else {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += base.raw(acc[i][j][e]);
      }
      sum *= base.fix;
#pragma unroll
      for (int d = 16; d < 64; d *= 2) sum += __shfl_xor(sum, d);
      if (lane < 16) sums[wa * (BP * 16) + (wb * T::kB + j) * 16 + lane] = make_float2(top, sum);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < BP * 16; c += 64 * WA * WB) {
      const int32_t tok = bb * BP * 16 + c;
      if (tok >= t.m16) continue;
      float2 r = sums[c];
#pragma unroll
      for (int a = 1; a < WA; ++a) {
        const float2 o = sums[a * (BP * 16) + c];
        const float top = o.x > r.x || o.x != o.x ? o.x : r.x;
        r = make_float2(top, r.y * rescale(r.x, top) + o.y * rescale(o.x, top));
      }
      t.part[(t.v0 / (16 * AP) + ab) * t.m16 + tok] = r;
    }
  } else {
    const float gtop = *t.gtop;
#pragma unroll
    for (int j = 0; j < T::kB; ++j) {
      const int32_t tok = tbase + 16 * j;
      const int64_t want = tok < t.m ? t.target[tok] : t.ignore;
      const bool seen = tok < t.m && want != t.ignore;
      const bool valid = want >= 0 && want < t.n_vocab;
      const ExpBase base(seen ? t.lse[tok] : 0.f);
      const float g = seen ? t.grad[tok] / gtop * g_scale<DT>() : 0.f;
      const float f = g * base.fix;
      if (__any(base.far)) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = base.raw_any(acc[i][j][e]) * f;
      } else {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = base.raw(acc[i][j][e]) * f;
      }
      // the few wavefronts that hold a target, a token that does not count or
      // has no valid target, or rows behind the vocabulary
      const int32_t at = place(want);
      if (__any(at >= 0)) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] -= at == 16 * i + e ? g : 0.f;
      }
      if (edge || __any(!seen || !valid)) {
#pragma unroll
        for (int i = 0; i < T::kA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!valid) acc[i][j][e] = __builtin_nanf("");
            if (!seen || 16 * i + e >= live) acc[i][j][e] = 0.f;
          }
      }
#pragma unroll
      for (int i = 0; i < T::kA; ++i) {
        // Row tok % 16 of panel tok / 16.  The four entries 16 i + 4 q + e,
        // q = lane / 16, lie where a lane of the dX product that reads W'
        // transposed holds the same rows of W' (hyb_panel.h): unit 2 (i % 2) +
        // q % 2, half q / 2 of its 16 bytes; of codes, rows in order, unit
        // 2 (i % 2) + q / 2, half q % 2.
        const int32_t col = (ab * AP + wa * T::kA + i) * 16;
        const int q = lane >> 4, half = is_f8(KIND) ? q & 1 : q >> 1;
        const int u = 2 * ((col >> 4) & 1) + (is_f8(KIND) ? q >> 1 : q & 1);
        if (tok < t.m16 && col < t.g_steps * 64)
          *reinterpret_cast<uint2*>(t.g + (int64_t(tok >> 4) * t.g_steps + (col >> 6)) * kPanelStep +
                                    ((col & 32) >> 5) * 1024 + u * 256 + (tok & 15) * 16 + half * 8) =
              round16x4<DT>(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      }
    }
  }
}

// Loss and lse of a token from its softmax sums and its target's logit.
__device__ __forceinline__ void store_loss(float2 sums, float z_target, int64_t want, int64_t ignore, int64_t n_vocab,
                                           float* loss, float* lse) {
  const float total = sums.x + logf(sums.y);
  if (want == ignore) {
    *loss = 0.f;
    *lse = 0.f;
  } else {
    *loss = want >= 0 && want < n_vocab ? total - z_target : __builtin_nanf("");
    *lse = total;
  }
}

// Softmax sums of rows of fp32 logits (the piece from t.v0, a multiple of a
// chunk), one workgroup per chunk of 256 EACH entries and token.  LAST: the one
// chunk is all of the vocabulary, and the loss follows at once (1024 x 512, 200
// tokens 4 us; two launches 3.7 + 3.4).  Bound by latency: the logits were just
// written and lie in the last-level cache (5 tokens x 32000 5 us).
template <int EACH, bool LAST>
__global__ __launch_bounds__(256) void k_xent_rows(const float* __restrict__ z, int64_t ldz, XentTile t,
                                                   float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 sums[4];
  __shared__ float z_target;
  const int32_t tok = int32_t(blockIdx.y);
  const int64_t v0 = t.v0 + int64_t(blockIdx.x) * (256 * EACH);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t want = t.target[tok];
  float v[EACH];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int64_t c = v0 + i * 256 + threadIdx.x;
    v[i] = c < t.n_vocab && c - t.v0 < ldz ? z[tok * ldz + c - t.v0] : -__builtin_inff();
    if (c == want && c < t.n_vocab) (LAST ? z_target : t.zt[tok]) = v[i];
    top = v[i] > top || v[i] != v[i] ? v[i] : top;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const float o = __shfl_xor(top, d);
    top = o > top || o != o ? o : top;
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EACH; ++i) sum += rescale(v[i], top) * (v[i] == -__builtin_inff() ? 0.f : 1.f);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  if (lane == 0) sums[wave] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 r = sums[0];
    for (int a = 1; a < 4; ++a) {
      const float2 o = sums[a];
      const float m = o.x > r.x || o.x != o.x ? o.x : r.x;
      r = make_float2(m, r.y * rescale(r.x, m) + o.y * rescale(o.x, m));
    }
    if constexpr (LAST)
      store_loss(r, z_target, want, t.ignore, t.n_vocab, loss + tok, lse + tok);
    else
      t.part[v0 / (256 * EACH) * t.m16 + tok] = r;
  }
}

// G of a piece from its logits (few tokens): one wavefront per 16 tokens and 64
// entries, in the order in which k_xent_tile leaves it.
template <int DT, bool F8>
__global__ __launch_bounds__(256) void k_xent_g_rows(const float* __restrict__ z, int64_t ldz, XentTile t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t s = int32_t(blockIdx.x) * 4 + wave;
  if (s >= t.g_steps) return;
  const int32_t tok = int32_t(blockIdx.y) * 16 + (lane & 15);
  const int64_t want = tok < t.m ? t.target[tok] : t.ignore;
  const bool seen = tok < t.m && want != t.ignore;
  const bool valid = want >= 0 && want < t.n_vocab;
  const float lse = seen ? t.lse[tok] : 0.f;
  const float f = seen ? t.grad[tok] / *t.gtop * g_scale<DT>() : 0.f;
  const int u = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint16_t g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = s * 64 + h * 32 + (F8 ? 8 * u + e : 16 * (u >> 1) + 4 * (u & 1) + 8 * (e >> 2) + (e & 3));
      const int64_t v = t.v0 + c;
      const float logit = seen && v < t.n_vocab ? z[tok * ldz + c] : 0.f;
      float p = (fast_exp(logit - lse) - (v == want ? 1.f : 0.f)) * f;
      if (!valid) p = __builtin_nanf("");
      if (!seen || v >= t.n_vocab) p = 0.f;
      g[e] = round16<DT>(p);
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = g[2 * e] | uint32_t(g[2 * e + 1]) << 16;
    *reinterpret_cast<uint4*>(t.g + (int64_t(blockIdx.y) * t.g_steps + s) * kPanelStep + h * 1024 + lane * 16) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Joins a token's partial sums: 16 tokens per workgroup, 64 threads each, in a
// fixed order (4096 tokens x 501 sums 9 us).
__global__ __launch_bounds__(1024) void k_xent_join(const float2* __restrict__ part, int64_t chunks, int32_t m,
                                                    int32_t m16, const float* __restrict__ zt,
                                                    const int64_t* __restrict__ target, int64_t ignore,
                                                    int64_t n_vocab, float* __restrict__ loss,
                                                    float* __restrict__ lse) {
  __shared__ float2 sums[64][16];
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int32_t tok = int32_t(blockIdx.x) * 16 + l;
  float2 r = make_float2(-__builtin_inff(), 0.f);
  auto join = [](float2 a, float2 o) {
    const float top = o.x > a.x || o.x != o.x ? o.x : a.x;
    return make_float2(top, a.y * rescale(a.x, top) + o.y * rescale(o.x, top));
  };
  if (tok < m)
    for (int64_t c = g; c < chunks; c += 64) r = join(r, part[c * m16 + tok]);
  sums[g][l] = r;
  for (int d = 32; d > 0; d /= 2) {
    __syncthreads();
    if (g < d) sums[g][l] = join(sums[g][l], sums[g + d][l]);
  }
  if (g == 0 && tok < m) {
    store_loss(sums[0][l], zt[tok], target[tok], ignore, n_vocab, loss + tok, lse + tok);
  }
}

// ------------------------------------------------------------ the gradients --

// Smallest power of two >= the largest finite |grad| of a token that counts
// (2^-100 if there is none); also clears *top.  One workgroup, 5 us.
__global__ __launch_bounds__(1024) void k_xent_grad_top(const float* __restrict__ grad,
                                                        const int64_t* __restrict__ target, int64_t ignore, int32_t m,
                                                        float* __restrict__ gtop, uint32_t* __restrict__ top) {
  __shared__ uint32_t tops[16];
  uint32_t u = 0;
  for (int32_t i = threadIdx.x; i < m; i += 1024) {
    const uint32_t b = __builtin_bit_cast(uint32_t, grad[i]) & 0x7FFFFFFFu;
    if (target[i] != ignore && b < 0x7F800000u && b > u) u = b;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_xor(u, d);
    u = o > u ? o : u;
  }
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = u;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) u = tops[i] > u ? tops[i] : u;
    u = (u + 0x7FFFFFu) & 0x7F800000u;
    // grad / gtop and the product with gtop stay in range: 2^-100 .. 2^100
    if (u < 0x0D800000u) u = 0x0D800000u;
    if (u > 0x71800000u) u = 0x71800000u;
    *gtop = __builtin_bit_cast(float, u);
    *top = 0;
  }
}

struct XentOut {
  float* acc;        // dX: [part][row][ld] fp32
  int64_t ld, part;  // floats
  int first;         // store (first piece) or add
  uint16_t* y;       // dW: 16-bit rows of the head's type
  int64_t ldy;
  const float* gtop;
  int32_t rows, cols;  // rows of B and columns (rows of A) that exist
  int64_t live;        // dW: rows from here on are padding, zero
};

// DX: Y[token, column] = sum over the piece's entries of G W' (A = W' read
// transposed, B = G), fp32, this workgroup's part of the steps, stored or
// added.  Else dW: Y[entry, column] = sum over tokens of G^T X (both read
// transposed), 16-bit, scaled back by gtop.  Bound as k_xent_tile is: a piece of
// 32768 x 4096 with 4096 tokens takes 835 us for dX, 819 for dW (1.3 PFLOP/s);
// dX over codes, 1000 tokens and 32768 x 5120, 291 us (1.15 PFLOP/s: 240
// workgroups, the vector unit widening beside the matrix unit).
template <int DT, bool DX, bool TILED, bool CODES, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void k_xent_product(PanelOperand A, PanelOperand B, int32_t steps,
                                                               int parts, XentOut o) {
  typedef PanelTile<DT, AP, BP, WA, WB, 2, true, !DX, TILED, CODES> T;
  extern __shared__ __attribute__((aligned(1024))) char xent_smem[];
  const int32_t na = (A.steps * (CODES ? 8 : 4) + AP - 1) / AP;
  const int32_t nb = DX ? (B.rows16 / 16 + BP - 1) / BP : (B.steps * 4 + BP - 1) / BP;
  int32_t ab, bb;
  const int32_t part = int32_t(blockIdx.y);
  panel_block(panel_order(int32_t(blockIdx.x), na * nb), na, nb, ab, bb);
  const int32_t quads = (steps + 3) / 4;  // a part is a whole number of four steps
  const int32_t s0 = int32_t(int64_t(quads) * part / parts) * 4;
  const int32_t s1 = part + 1 == parts ? steps : int32_t(int64_t(quads) * (part + 1) / parts) * 4;
  f32x4_t acc[T::kA][T::kB];
  T::run(A, B, ab * AP, bb * BP, s0, s1, xent_smem, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave % WA, wb = wave / WA;
  if constexpr (DX) {
#pragma unroll
    for (int j = 0; j < T::kB; ++j) {
      const int32_t row = (bb * BP + wb * T::kB + j) * 16 + (lane & 15);
      if (row >= o.rows) continue;
#pragma unroll
      for (int i = 0; i < T::kA; ++i) {
        const int32_t col = (ab * AP + wa * T::kA + i) * 16 + (lane >> 4) * 4;
        if (col >= o.ld) continue;
        f32x4_t* p = reinterpret_cast<f32x4_t*>(o.acc + part * o.part + row * o.ld + col);
        f32x4_t v = acc[i][j];
        if (!o.first) {
          const f32x4_t u = *p;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += u[e];
        }
        *p = v;
      }
    }
  } else {
    const float back = *o.gtop / g_scale<DT>();
    // G's entries 4..7 and 8..11 of 16 have changed places
    const int row16 = (lane & 3) | (lane & 4) << 1 | (lane & 8) >> 1;
    const int32_t row0 = (bb * BP + wb * T::kB) * 16, col0 = (ab * AP + wa * T::kA) * 16;
    __syncthreads();  // the tile's LDS stages are free
    panel_rows16<T::kA, T::kB>(
        xent_smem + wave * (T::kA * T::kB * 512), lane, row16,
        [&](int i, int j) {
          const bool live = row0 + j * 16 + row16 < o.live;
          const f32x4_t v = acc[i][j];
          const uint2 h = round16x4<DT>(v[0] * back, v[1] * back, v[2] * back, v[3] * back);
          return live ? h : make_uint2(0, 0);
        },
        [&](int r, int c, uint4 u) {
          const int32_t row = row0 + r, col = col0 + c;  // a packed head's k is a multiple of 64
          if (row < o.rows && col < o.cols)
            *reinterpret_cast<Bytes16*>(o.y + row * o.ldy + col) = Bytes16{{u.x, u.y, u.z, u.w}};
        });
  }
}

// dX = gtop * sum of the parts (in order), rounded once; ignored tokens 0.  Bound
// by memory (4096 x 4096, one part, 22 us).
template <int DT, bool F8>
__global__ __launch_bounds__(256) void k_xent_dx(const float* __restrict__ acc, int64_t ld, int64_t part, int parts,
                                                 int32_t m, int32_t k, const int64_t* __restrict__ target,
                                                 int64_t ignore, const float* __restrict__ gtop,
                                                 const uint32_t* __restrict__ top, uint16_t* __restrict__ dx,
                                                 int64_t lddx) {
  const int64_t tok = blockIdx.x;
  const int32_t col = (int32_t(blockIdx.y) * 256 + threadIdx.x) * 4;
  if (col >= k) return;
  const bool seen = target[tok] != ignore;
  f32x4_t v = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (seen) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const f32x4_t u = *reinterpret_cast<const f32x4_t*>(acc + p * part + tok * ld + col);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    }
    const float f = *gtop / g_scale<DT>();
    // the fp16 form of an 8-bit head was divided by 2^(top - 133)
    const int lift = F8 && DT == HYB_F16 ? int(*top) - 133 : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e] * f, lift);
  }
  uint16_t* p = dx + tok * lddx + col;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < k) p[e] = round16<DT>(v[e]);
}

// dW of an empty batch.
__global__ __launch_bounds__(256) void k_xent_zero(uint16_t* __restrict__ dw, int64_t n, int64_t ld, int32_t k) {
  const int32_t c = int32_t(blockIdx.y) * 256 + threadIdx.x;
  for (int64_t r = blockIdx.x; r < n; r += gridDim.x)
    if (c < k) dw[r * ld + c] = 0;
}

// ----------------------------------------------------------------- launches --

template <typename F>
hipError_t allow_lds(F* fn, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int KIND, int DT, bool GRAD, bool TILED, int AP, int BP, int WA, int WB>
hipError_t run_tile(const PanelOperand& W, const PanelOperand& X, const XentTile& t, hipStream_t s) {
  typedef PanelTile<KIND, AP, BP, WA, WB, 2, false, false, TILED> T;
  const hipError_t e = allow_lds(&k_xent_tile<KIND, DT, GRAD, TILED, AP, BP, WA, WB>, T::kLds);
  if (e != hipSuccess) return e;
  const int64_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  hipLaunchKernelGGL((k_xent_tile<KIND, DT, GRAD, TILED, AP, BP, WA, WB>), dim3(unsigned(na * nb)), dim3(64 * WA * WB),
                     T::kLds, s, W, X, t);
  return hipGetLastError();
}

template <int KIND, int DT, bool GRAD, bool TILED>
hipError_t run_shape(int bp, const PanelOperand& W, const PanelOperand& X, const XentTile& t, hipStream_t s) {
  // (4 goes with up to 64 tokens, whose logits come from the library's product)
  if (bp == 16) return run_tile<KIND, DT, GRAD, TILED, 16, 16, 2, 4>(W, X, t, s);
  return run_tile<KIND, DT, GRAD, TILED, 16, 8, 4, 2>(W, X, t, s);
}

template <int DT, bool GRAD>
hipError_t run_tiles(const XentPlan& p, const PanelOperand& W, const PanelOperand& X, const XentTile& t,
                     hipStream_t s) {
  return p.f8 ? run_shape<kF8Wide, DT, GRAD, false>(p.bp, W, X, t, s) : run_shape<DT, DT, GRAD, true>(p.bp, W, X, t, s);
}

template <int DT, bool DX, bool TILED, bool CODES, int AP, int BP, int WA, int WB>
hipError_t run_product(const PanelOperand& A, const PanelOperand& B, int32_t steps, int parts, const XentOut& o,
                       hipStream_t s) {
  typedef PanelTile<DT, AP, BP, WA, WB, 2, true, !DX, TILED, CODES> T;
  const hipError_t e = allow_lds(&k_xent_product<DT, DX, TILED, CODES, AP, BP, WA, WB>, T::kLds);
  if (e != hipSuccess) return e;
  const int64_t na = (A.steps * (CODES ? 8 : 4) + AP - 1) / AP;
  const int64_t nb = DX ? (B.rows16 / 16 + BP - 1) / BP : (B.steps * 4 + BP - 1) / BP;
  hipLaunchKernelGGL((k_xent_product<DT, DX, TILED, CODES, AP, BP, WA, WB>), dim3(unsigned(na * nb), unsigned(parts)),
                     dim3(64 * WA * WB), T::kLds, s, A, B, steps, parts, o);
  return hipGetLastError();
}

template <int DT, bool F8>
hipError_t run_dx(int bp, const PanelOperand& A, const PanelOperand& B, int32_t steps, int parts, const XentOut& o,
                  hipStream_t s) {
  // (codes: the more wavefronts along the columns, the fewer convert the same
  // one; at eight of them the 128-token tile needs 150 registers, which leaves one
  // workgroup a compute unit: 100 tokens, 128256 x 4096 215 us against 128)
  if (bp == 16) return run_product<DT, true, !F8, F8, 16, 16, F8 ? 4 : 2, F8 ? 2 : 4>(A, B, steps, parts, o, s);
  if (bp == 8) return run_product<DT, true, !F8, F8, 16, 8, 4, 2>(A, B, steps, parts, o, s);
  return run_product<DT, true, !F8, F8, 16, 4, F8 ? 8 : 4, F8 ? 1 : 2>(A, B, steps, parts, o, s);
}

// The tile rows of a piece that were expanded (PanelOperand): none by default.
struct Spare {
  const char* at = nullptr;
  int32_t first = 0, end = 0;
};

// The tiles of the piece of `rows` vocabulary rows from v0 that PanelOperand
// calls spare, in `out`: over sparse tiles those of every tile row, else the one
// tile row that the vocabulary ends within (tiles behind it, and ones without a
// slot, read as zeros).
hipError_t prepare_piece(const hyb_head& head, const XentPlan& p, int64_t n_vocab, int64_t plain, int64_t v0,
                         int64_t rows, char* out, Spare* spare, hipStream_t s) {
  const hyb_layout& L = *head.layout;
  const hyb_packed& P = *head.packed;
  int64_t from = v0, end = v0 + rows;
  if (L.n_sparse == 0) {
    from = n_vocab / L.b1 * L.b1;
    if (from == n_vocab || from < v0 || from >= end) return hipSuccess;
    if (end > from + L.b1) end = from + L.b1;
  }
  *spare = Spare{out, int32_t((from - v0) / L.b1), int32_t((end - v0 + L.b1 - 1) / L.b1)};
  const unsigned panels = unsigned((end - from + 15) / 16);
  hipLaunchKernelGGL(k_xent_expand, dim3(panels, unsigned((p.steps + 3) / 4)), dim3(256), 0, s,
                     static_cast<const uint4*>(P.dense), static_cast<const uint4*>(P.val),
                     static_cast<const uint16_t*>(P.meta), P.tidx, L.b1, L.b2, L.meta, int32_t(L.tiles_k),
                     int32_t(L.n_dense), int32_t(L.n_sparse), from, n_vocab, plain, int32_t(p.steps), out);
  return hipGetLastError();
}

// x as the B operand of the logits product.
hipError_t prepare_x(const XentPlan& p, const void* x, int dtype, int64_t ldx, const int64_t* target, int64_t ignore,
                     char* ws, hipStream_t s, PanelOperand* out) {
  if (p.f8) {
    const hyb_f8 X{ws + p.x, ws + p.xs};
    *out = PanelOperand{ws + p.x, int32_t(p.m16), int32_t(p.steps), reinterpret_cast<const uint32_t*>(ws + p.xs), p.m16};
    return launch_f8_quantize(x, dtype, p.m, p.k, ldx, HYB_F8_ROWS, X, s);
  }
  *out = PanelOperand{ws + p.x, int32_t(p.m16), int32_t(p.steps), nullptr, 0};
  hipLaunchKernelGGL(k_xent_pack_x, dim3(unsigned(p.m16 / 16), unsigned((p.steps + 3) / 4)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(x), ldx, p.m, int32_t(p.steps), target, ignore, ws + p.x);
  return hipGetLastError();
}

// The A operand of the logits product for a piece.
PanelOperand piece_operand(const hyb_head& head, const XentPlan& p, int64_t plain, int64_t v0, int64_t rows,
                           const Spare& spare) {
  PanelOperand o{};
  o.rows16 = int32_t((rows + 15) / 16 * 16);
  o.steps = int32_t(p.steps);
  if (p.f8) {
    o.data = static_cast<const char*>(head.f8->codes) + v0 / 16 * p.steps * kPanelStep;
    o.scale = static_cast<const uint32_t*>(head.f8->scales) + v0;
    o.scale_pitch = f8_rows16(p.n);
    return o;
  }
  const hyb_layout& L = *head.layout;
  o.data = static_cast<const char*>(head.packed->dense);
  o.log_b1 = __builtin_ctz(L.b1);
  o.log_b2 = __builtin_ctz(L.b2);
  o.tiles_k = int32_t(L.tiles_k);
  o.n_dense = int32_t(L.n_dense);
  o.row0 = v0;
  o.plain = plain;
  o.tidx = head.packed->tidx;
  o.spare = spare.at;
  o.spare0 = spare.first;
  o.spare1 = spare.end;
  return o;
}

#define HYB_TRY(call)                      \
  do {                                     \
    const hipError_t e_ = (call);          \
    if (e_ != hipSuccess) return e_;       \
  } while (0)

// Logits of the vocabulary rows v0 .. v0 + rows - 1 (few tokens) through the
// library's products, fp32, row stride ldz; an 8-bit head multiplies the
// quantised x of prepare_x.  The products get no workspace: where their route
// would cut k, its tile runs over all of k.
hipError_t piece_logits(const hyb_head& head, const XentPlan& p, const void* x, int64_t ldx, int64_t v0, int64_t rows,
                        float* z, int64_t ldz, char* ws, hipStream_t s) {
  if (p.f8) {
    const hyb_f8 W{static_cast<char*>(head.f8->codes) + v0 / 16 * p.steps * kPanelStep,
                   static_cast<uint32_t*>(head.f8->scales) + v0};
    return launch_f8_gemm(W, rows, p.k, hyb_f8{ws + p.x, ws + p.xs}, p.m, z, HYB_F32, ldz, nullptr, s, f8_rows16(p.n));
  }
  // the piece's tile rows: the same streams, a part of the tile index
  hyb_layout L = *head.layout;
  hyb_packed P = *head.packed;
  P.tidx += v0 / L.b1 * L.tiles_k;
  L.n = rows;
  L.tiles_n = rows / L.b1;
  if (p.m <= kGemvCrossoverM || (p.m <= kMaxGemvM && gemv_preferred(L, int(p.m))))
    return launch_gemv(L, P, x, int(p.m), ldx, z, HYB_F32, ldz, s);
  return launch_gemm(L, P, x, int(p.m), ldx, z, HYB_F32, ldz, s, nullptr, 0);
}

template <int DT>
hipError_t loss_typed(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int64_t ldx, XentTile t,
                      float* loss, float* lse, char* ws, hipStream_t s) {
  int64_t chunks = 0;
  if (p.rows) {
    float* z = reinterpret_cast<float*>(ws + p.logits);
    if (p.f8) {
      PanelOperand X;
      HYB_TRY(prepare_x(p, x, DT, ldx, t.target, t.ignore, ws, s, &X));
    }
    for (int64_t v0 = 0; v0 < n_vocab; v0 += p.at_once) {
      const int64_t rows = p.n - v0 < p.at_once ? p.n - v0 : p.at_once;
      const int64_t ldz = (rows + 3) / 4 * 4;
      HYB_TRY(piece_logits(head, p, x, ldx, v0, rows, z, ldz, ws, s));
      t.v0 = v0;
      const int64_t live = n_vocab - v0 < rows ? n_vocab - v0 : rows;
      if (n_vocab <= 8192) {  // (one piece)
        const dim3 grid(1, unsigned(p.m));
        if (n_vocab <= 2048)
          hipLaunchKernelGGL((k_xent_rows<8, true>), grid, dim3(256), 0, s, z, ldz, t, loss, lse);
        else
          hipLaunchKernelGGL((k_xent_rows<32, true>), grid, dim3(256), 0, s, z, ldz, t, loss, lse);
        return hipGetLastError();
      }
      hipLaunchKernelGGL((k_xent_rows<8, false>), dim3(unsigned((live + 2047) / 2048), unsigned(p.m)), dim3(256), 0, s, z,
                         ldz, t, loss, lse);
      HYB_TRY(hipGetLastError());
      chunks = (v0 + live + 2047) / 2048;
    }
  } else {
    PanelOperand X;
    HYB_TRY(prepare_x(p, x, DT, ldx, t.target, t.ignore, ws, s, &X));
    // (Logits of padding rows are not looked at: no tile row is spare for them.)
    const bool expand = !p.f8 && head.layout->n_sparse > 0;
    for (int64_t v0 = 0; v0 < n_vocab; v0 += p.at_once) {
      const int64_t rows = n_vocab - v0 < p.at_once ? n_vocab - v0 : p.at_once;
      Spare spare;
      if (expand) HYB_TRY(prepare_piece(head, p, n_vocab, p.n, v0, rows, ws + p.w, &spare, s));
      t.v0 = v0;
      const PanelOperand W = piece_operand(head, p, p.n, v0, rows, spare);
      HYB_TRY((run_tiles<DT, false>(p, W, X, t, s)));
      chunks = v0 / 256 + (W.rows16 + 255) / 256;
    }
  }
  hipLaunchKernelGGL(k_xent_join, dim3(unsigned(p.m16 / 16)), dim3(1024), 0, s, t.part, chunks, t.m, t.m16, t.zt,
                     t.target, t.ignore, n_vocab, loss, lse);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_typed(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int64_t ldx,
                          XentTile t, void* dx, int64_t lddx, void* dw, int64_t lddw, char* ws, hipStream_t s) {
  float* gtop = reinterpret_cast<float*>(ws + p.misc);
  uint32_t* top = reinterpret_cast<uint32_t*>(ws + p.misc + 64);
  hipLaunchKernelGGL(k_xent_grad_top, dim3(1), dim3(1024), 0, s, t.grad, t.target, t.ignore, t.m, gtop, top);
  HYB_TRY(hipGetLastError());
  t.gtop = gtop;
  if (p.f8 && dx && DT == HYB_F16) {
    hipLaunchKernelGGL(k_xent_top_scale, dim3(unsigned((n_vocab + 255) / 256), unsigned((p.steps + 3) / 4)), dim3(256),
                       0, s, static_cast<const uint32_t*>(head.f8->scales), f8_rows16(p.n), n_vocab, int32_t(p.steps),
                       top);
    HYB_TRY(hipGetLastError());
  }
  PanelOperand X{};
  if (p.f8 || !p.rows || dw) HYB_TRY(prepare_x(p, x, DT, ldx, t.target, t.ignore, ws, s, &X));
  const int32_t krows = int32_t(p.ksteps16 * 64);
  t.g = ws + p.g;
  // dX runs over the vocabulary that counts, dW over every row of the head.
  const int64_t end = dw ? p.n : n_vocab;
  for (int64_t v0 = 0; v0 < end; v0 += p.at_once) {
    const int64_t rows = end - v0 < p.at_once ? end - v0 : p.at_once;
    const int32_t vsteps = int32_t((rows + 63) / 64);
    t.v0 = v0;
    t.g_steps = vsteps;
    // (the logits of few tokens do not need them)
    Spare spare;
    if (!p.f8 && (!p.rows || dx)) HYB_TRY(prepare_piece(head, p, n_vocab, n_vocab, v0, rows, ws + p.w, &spare, s));
    PanelOperand W = piece_operand(head, p, n_vocab, v0, rows, spare);
    if (p.f8) {
      W.plain = n_vocab - v0;
      W.top = top;
    }
    if (p.rows) {
      // all of a packed head's tile rows that the piece's vocabulary reaches into
      // (not its padding: a product of other rows may take another route, and dX
      // would differ in its last bits with and without dW)
      const int64_t live = n_vocab - v0 < rows ? n_vocab - v0 : rows;
      const int64_t b1 = p.f8 ? 1 : head.layout->b1, whole = (live + b1 - 1) / b1 * b1, ldz = (whole + 3) / 4 * 4;
      float* z = reinterpret_cast<float*>(ws + p.logits);
      if (live > 0) HYB_TRY(piece_logits(head, p, x, ldx, v0, whole, z, ldz, ws, s));
      const dim3 grid(unsigned((vsteps + 3) / 4), unsigned(p.m16 / 16));
      if (p.f8)
        hipLaunchKernelGGL((k_xent_g_rows<DT, true>), grid, dim3(256), 0, s, z, ldz, t);
      else
        hipLaunchKernelGGL((k_xent_g_rows<DT, false>), grid, dim3(256), 0, s, z, ldz, t);
      HYB_TRY(hipGetLastError());
    } else {
      HYB_TRY((run_tiles<DT, true>(p, W, X, t, s)));
    }
    // G: tokens x entries, vsteps steps; W': entries x columns
    const PanelOperand G{ws + p.g, int32_t(p.m16), vsteps, nullptr, 0};
    if (dx && v0 < n_vocab) {
      // (the steps of the vocabulary, so that dX does not depend on whether dW
      // is asked for)
      const int32_t dx_steps = int32_t(((n_vocab - v0 < rows ? n_vocab - v0 : rows) + 63) / 64);
      XentOut o{};
      o.acc = reinterpret_cast<float*>(ws + p.dx);
      o.ld = krows;
      o.part = p.m * int64_t(krows);
      o.first = v0 == 0;
      o.rows = int32_t(p.m);
      o.cols = krows;
      HYB_TRY(p.f8 ? (run_dx<DT, true>(p.bp, W, G, dx_steps, p.parts, o, s))
                   : (run_dx<DT, false>(p.bp, W, G, dx_steps, p.parts, o, s)));
    }
    if (dw) {
      XentOut o{};
      o.y = static_cast<uint16_t*>(dw) + v0 * lddw;
      o.ldy = lddw;
      o.gtop = gtop;
      o.rows = int32_t(rows);
      o.cols = int32_t(p.k);
      o.live = n_vocab - v0;
      // few tokens: bound by the writes of dW, and two of the smaller tiles share
      // a CU (65536 x 4096, 16 / 200 / 400 / 800 tokens, logits included: 340 /
      // 505 / 601 / 998 us against 386 / 537 / 603 / 956)
      HYB_TRY(p.m <= 256 ? (run_product<DT, false, false, false, 8, 8, 2, 4>(X, G, int32_t(p.m64 / 64), 1, o, s))
                         : (run_product<DT, false, false, false, 16, 16, 2, 4>(X, G, int32_t(p.m64 / 64), 1, o, s)));
    }
  }
  if (dx) {
    const dim3 grid(unsigned(p.m), unsigned((p.k + 1023) / 1024));
    const float* acc = reinterpret_cast<const float*>(ws + p.dx);
    if (p.f8)
      hipLaunchKernelGGL((k_xent_dx<DT, true>), grid, dim3(256), 0, s, acc, int64_t(krows), p.m * int64_t(krows),
                         p.parts, t.m, int32_t(p.k), t.target, t.ignore, gtop, top, static_cast<uint16_t*>(dx), lddx);
    else
      hipLaunchKernelGGL((k_xent_dx<DT, false>), grid, dim3(256), 0, s, acc, int64_t(krows), p.m * int64_t(krows),
                         p.parts, t.m, int32_t(p.k), t.target, t.ignore, gtop, top, static_cast<uint16_t*>(dx), lddx);
    HYB_TRY(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_xent(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int dtype, int64_t ldx,
                       const int64_t* target, int64_t ignore, float* loss, float* lse, char* ws, hipStream_t s) {
  XentTile t{};
  t.n_vocab = n_vocab;
  t.ignore = ignore;
  t.target = target;
  t.m = int32_t(p.m);
  t.m16 = int32_t(p.m16);
  t.part = reinterpret_cast<float2*>(ws + p.part);
  t.zt = reinterpret_cast<float*>(ws + p.zt);
  return dtype == HYB_BF16 ? loss_typed<HYB_BF16>(head, p, n_vocab, x, ldx, t, loss, lse, ws, s)
                           : loss_typed<HYB_F16>(head, p, n_vocab, x, ldx, t, loss, lse, ws, s);
}

hipError_t launch_xent_backward(const hyb_head& head, const XentPlan& p, int64_t n_vocab, const void* x, int dtype,
                                int64_t ldx, const int64_t* target, int64_t ignore, const float* lse,
                                const float* grad, void* dx, int64_t lddx, void* dw, int64_t lddw, char* ws,
                                hipStream_t s) {
  if (p.m == 0) {
    hipLaunchKernelGGL(k_xent_zero, dim3(unsigned(p.n < 4096 ? p.n : 4096), unsigned((p.k + 255) / 256)), dim3(256), 0,
                       s, static_cast<uint16_t*>(dw), p.n, lddw, int32_t(p.k));
    return hipGetLastError();
  }
  XentTile t{};
  t.n_vocab = n_vocab;
  t.ignore = ignore;
  t.target = target;
  t.m = int32_t(p.m);
  t.m16 = int32_t(p.m16);
  t.lse = lse;
  t.grad = grad;
  return dtype == HYB_BF16 ? backward_typed<HYB_BF16>(head, p, n_vocab, x, ldx, t, dx, lddx, dw, lddw, ws, s)
                           : backward_typed<HYB_F16>(head, p, n_vocab, x, ldx, t, dx, lddx, dw, lddw, ws, s);
}

}  // namespace hyb
