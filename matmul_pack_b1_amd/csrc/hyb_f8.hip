// Kernels of the 8-bit block-scaled matrices (include/hyb_f8.h): quantise,
// read back, and the product on the scaled matrix instructions.
#include <type_traits>

#include "hyb_f8_internal.h"
#include "hyb_panel.h"

namespace hyb {
namespace {

// ------------------------------------------------------ quantise, read back --

// Eight columns c0.. of one row, as loaded: two elements to a word, or one
// for fp32 (k = 0: no row, zeros).
template <int DT>
struct Eight {
  uint32_t w[DT == HYB_F32 ? 8 : 4];
};

// A lane at or behind the row's end loads the row's last eight columns, so
// that a wavefront's loads of many rows need no branches and are all under
// way at once; trim8 then moves its columns into place and zeros the rest.
template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void* a, int64_t base, int32_t c0, int32_t k) {
  Eight<DT> r;
  constexpr int kWords = DT == HYB_F32 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < kWords; ++i) r.w[i] = 0;
  if (k == 0) return r;
  if (k < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < k) {
        if constexpr (DT == HYB_F32)
          r.w[i] = static_cast<const uint32_t*>(a)[base + c0 + i];
        else
          r.w[i / 2] |= uint32_t(static_cast<const uint16_t*>(a)[base + c0 + i]) << (16 * (i & 1));
      }
    return r;
  }
  const int64_t at = base + (c0 < k - 8 ? c0 : k - 8);
  const Bytes16* p = reinterpret_cast<const Bytes16*>(static_cast<const char*>(a) + at * (DT == HYB_F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i) {
    const Bytes16 u = p[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[4 * i + j] = u.w[j];
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void trim8(Eight<DT>& r, int32_t c0, int32_t k) {
  if (k < 8) return;
  const int32_t by = c0 - (k - 8);  // columns to move down, 8 or more: none left
  constexpr int kWords = DT == HYB_F32 ? 8 : 4;
  auto move = [&](bool on, int words) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t u = i + words < kWords ? r.w[i + words < kWords ? i + words : 0] : 0;
      r.w[i] = on ? u : r.w[i];
    }
  };
  if constexpr (DT == HYB_F32) {
    move(by > 0 && (by & 4), 4);
    move(by > 0 && (by & 2), 2);
    move(by > 0 && (by & 1), 1);
  } else {
    move(by > 0 && (by & 4), 2);
    move(by > 0 && (by & 2), 1);
    const bool half = by > 0 && (by & 1);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t u = r.w[i] >> 16 | (i + 1 < kWords ? r.w[i + 1 < kWords ? i + 1 : 0] << 16 : 0);
      r.w[i] = half ? u : r.w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kWords; ++i) r.w[i] = by >= 8 ? 0 : r.w[i];
}

// Element i as fp32.
template <int DT>
__device__ __forceinline__ float elem(const Eight<DT>& r, int i) {
  if constexpr (DT == HYB_F32) return __builtin_bit_cast(float, r.w[i]);
  return widen16<DT>((r.w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
}

constexpr uint32_t kF32Inf = 0x7F800000u;

// fp32 bits of the largest magnitude; a NaN or an infinity gives at least
// kF32Inf.  (Magnitudes of one type order as their bits.)
template <int DT>
__device__ __forceinline__ uint32_t top_of(const Eight<DT>& r) {
  if constexpr (DT == HYB_F32) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = r.w[i] & 0x7FFFFFFFu;
      t = u > t ? u : t;
    }
    return t;
  } else {
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
    u16x2_t t = __builtin_bit_cast(u16x2_t, r.w[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2_t, r.w[i] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, widen16<DT>(t[0] > t[1] ? t[0] : t[1]));
  }
}

// The same over finite elements only.
template <int DT>
__device__ __forceinline__ uint32_t top_finite(const Eight<DT>& r) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, elem<DT>(r, i)) & 0x7FFFFFFFu;
    t = u < kF32Inf && u > t ? u : t;
  }
  return t;
}

// Largest of the 16 lanes of a row of lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xF, 0xF, false));  // row_ror:8
  v = o > v ? o : v;
  o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xF, 0xF, false));
  v = o > v ? o : v;
  o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x122, 0xF, 0xF, false));
  v = o > v ? o : v;
  o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x121, 0xF, 0xF, false));
  return o > v ? o : v;
}

// Exponent byte of a block whose largest finite magnitude has the bits
// `top`: 448 = 1.75 * 2^8, so with top = f * 2^p, 1 <= f < 2, the smallest
// exponent is p - 8 for f <= 1.75 and p - 7 above.  Magnitudes below the
// smallest normal number end at the smallest exponent, -127.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  if (top == 0) return 127u;
  const int p = int(top >> 23);  // biased; 0: subnormal
  const int e = p - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return uint32_t(e < 0 ? 0 : e);
}

// 2^(byte - 127) and its inverse; the ends of the range are subnormal.
__device__ __forceinline__ float exp2_byte(uint32_t byte) {
  return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
}

// Eight codes of a / 2^(e - 127); `mark` makes elements that are not finite
// the NaN code (the conversion is only given finite ones).
template <int DT>
__device__ __forceinline__ uint2 codes8(const Eight<DT>& r, uint32_t e, bool mark) {
  const float inv = exp2_byte(254u - e);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(elem<DT>(r, 4 * i) * inv, elem<DT>(r, 4 * i + 1) * inv, 0, false);
    w[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(elem<DT>(r, 4 * i + 2) * inv, elem<DT>(r, 4 * i + 3) * inv, lo, true));
    if (mark) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((__builtin_bit_cast(uint32_t, elem<DT>(r, 4 * i + j)) & 0x7FFFFFFFu) >= kF32Inf) w[i] |= 0xFFu << (8 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

// One wavefront per panel and step: a load covers 128 columns of four rows (8
// columns per lane, 16 lanes to a row), so a row's maximum is one over 16
// lanes, and a lane's codes are half of its row's 16 bytes of a unit, which
// leave as they are, in pieces of 64 bytes.  A workgroup takes four steps of a
// panel, or (a weight) one step of the eight panels of a block, whose maxima
// meet in LDS.  Bound by memory: one read of the matrix, half or a quarter as
// many bytes written.  28672 x 8192 bf16 as a weight 162 us (706 MB, 4.4 TB/s; a
// copy runs at 4.8), 2048 x 17408 as rows 18 us (6 TB/s, from the last-level
// cache); few rows by latency: one token of 4096 3.3 us, 256 of 5120 4.4.  (Four
// steps to a wavefront, through LDS into whole 1 KiB stores: 182, 20, 3.8, 9.1.)
template <int DT, bool WEIGHT>
__global__ __launch_bounds__(WEIGHT ? 512 : 256) void k_f8_quantize(const void* __restrict__ a, int64_t rows,
                                                                    int32_t k, int64_t lda, char* __restrict__ codes,
                                                                    char* __restrict__ scales, int32_t panels,
                                                                    int32_t steps, int32_t across) {
  __shared__ uint32_t top_lds[8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t id = int32_t(blockIdx.x), down = id / across, over = id % across;
  const int64_t panel = WEIGHT ? int64_t(down) * 8 + wave : down;
  const int32_t s = WEIGHT ? over : over * 4 + wave;
  const int64_t r0 = panel * 16;
  const int g = lane >> 4, j = lane & 15;
  const int32_t c0 = s * 128 + j * 8;
  const bool live = panel < panels && s < steps;
  Eight<DT> v[4];
  uint32_t top[4];
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = r0 + i * 4 + g;
    v[i] = load8<DT>(a, row * lda, c0, row < rows && live ? k : 0);
  }
  if (!__all(c0 + 8 <= k)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) trim8<DT>(v[i], c0, r0 + i * 4 + g < rows && live ? k : 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top[i] = top_of<DT>(v[i]);
    all = top[i] > all ? top[i] : all;
  }
  const bool mark = __any(all >= kF32Inf);
  if (mark) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = top_finite<DT>(v[i]);
  }
  if constexpr (WEIGHT) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = top[i] > t ? top[i] : t;
    t = max16(t);
#pragma unroll
    for (int d = 16; d < 64; d *= 2) {
      const uint32_t o = __shfl_xor(t, d);
      t = o > t ? o : t;
    }
    if (lane == 0) top_lds[wave] = t;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) t = top_lds[w] > t ? top_lds[w] : t;
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = t;
  }
  if (panel >= panels) return;
  // Columns 8 j.. of a step: half j / 8, unit (j % 8) / 2, one half of the
  // row's 16 bytes.
  char* out = codes + (panel * steps + s) * kPanelStep + (j >> 1) * 256 + (j & 1) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 4 + g;
    if constexpr (!WEIGHT) top[i] = max16(top[i]);
    const bool in = live && r0 + r < rows;
    const uint32_t e = in ? block_exponent(top[i]) : 127u;
    const uint2 u = codes8<DT>(v[i], e, mark);
    if (live) *reinterpret_cast<uint2*>(out + r * 16) = u;
    if (j == 0) scales[((int64_t(s >> 2) * panels * 16) + r0 + r) * 4 + (s & 3)] = char(e);
  }
}

// One wavefront per panel and step (a workgroup's four take four steps): its
// 1 KiB loads are the panel's order, its stores 16 columns of 16 rows.  Bound by
// memory: 28672 x 8192 to bf16 143 us (4.9 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void k_f8_dequantize(const char* __restrict__ codes,
                                                       const uint32_t* __restrict__ scales, int64_t rows, int32_t k,
                                                       int64_t lda, void* __restrict__ a, int32_t panels,
                                                       int32_t steps) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = blockIdx.x;
  const int64_t row = panel * 16 + (lane & 15);
  const int32_t s = int32_t(blockIdx.y) * 4 + wave;
  if (row >= rows || s >= steps) return;
  const uint32_t byte = (scales[int64_t(blockIdx.y) * panels * 16 + row] >> (8 * wave)) & 0xFFu;
  uint4 u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    u[h] = *reinterpret_cast<const uint4*>(codes + (panel * steps + s) * kPanelStep + h * 1024 + lane * 16);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t c0 = s * 128 + h * 64 + (lane >> 4) * 16;
    if (c0 >= k) continue;
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
    constexpr int kWords = DT == HYB_F32 ? 16 : 8;
    uint32_t o[kWords];
    if constexpr (DT == HYB_BF16) {
      // reads only the exponent of its scale; exact
      const float f = __builtin_bit_cast(float, byte << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], f, false));
        o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], f, true));
      }
    } else {
      const float scale = exp2_byte(byte);
      float f[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[4 * i] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 0) * scale;
        f[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 1) * scale;
        f[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 2) * scale;
        f[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 3) * scale;
      }
      if constexpr (DT == HYB_F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __builtin_bit_cast(uint32_t, f[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = round16<DT>(f[2 * i]) | uint32_t(round16<DT>(f[2 * i + 1])) << 16;
      }
    }
    const int64_t at = row * lda + c0;
    if (c0 + 16 <= k) {
      Bytes16* p = reinterpret_cast<Bytes16*>(static_cast<char*>(a) + at * (DT == HYB_F32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) p[i] = Bytes16{{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]}};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c0 + i < k) {
          if constexpr (DT == HYB_F32)
            static_cast<uint32_t*>(a)[at + i] = o[i];
          else
            static_cast<uint16_t*>(a)[at + i] = uint16_t(o[i / 2] >> (16 * (i & 1)));
        }
    }
  }
}

// ------------------------------------------------------------------ product --

struct F8Out {
  void* y;
  int64_t ldy;
  int32_t n, m, ydt;
};

// Four outputs n..n+3 of token m.
__device__ __forceinline__ void f8_store4(const F8Out& o, int64_t m, int32_t n, f32x4_t v) {
  if (m >= o.m || n >= o.n) return;
  const int64_t at = m * o.ldy + n;
  if (n + 4 <= o.n) {
    if (o.ydt == HYB_F32) {
      Bytes16 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = v[e];  // (a bit cast of a vector's element reads element 0)
        u.w[e] = __builtin_bit_cast(uint32_t, f);
      }
      *reinterpret_cast<Bytes16*>(static_cast<float*>(o.y) + at) = u;
    } else {
      const uint2 h = o.ydt == HYB_BF16 ? round16x4<HYB_BF16>(v[0], v[1], v[2], v[3])
                                        : round16x4<HYB_F16>(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<Bytes8*>(static_cast<uint16_t*>(o.y) + at) = Bytes8{{h.x, h.y}};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < o.n) store_out(o.y, o.ydt, at + e, v[e]);
}

// Few tokens: one w panel (16 rows) and BP x panels per workgroup, whose
// WAVES wavefronts take four steps (512 columns) in turn, the codes straight
// from memory to the operand registers.  Bound by the read of w, so the wide
// kind costs nothing here and serves every output type: 14336x4096 12.8 us at 1
// to 8 quantised tokens, 17408x5120 18.9 (4.7 TB/s).
//
// XDT other than 0 (BP 1, at most kFusedTokens tokens): X is still in its own
// type, and every wavefront quantises the columns it multiplies, while its
// codes of w are on their way.  Per token that costs every wavefront about 60
// instructions per four steps, a launch of its own 3 us once.  In one launch
// against two, at 1 / 2 / 4 tokens: 14336x4096 12.0 / 13.3 / 16.4 us against
// 15.5 / 15.7 / 15.7, 5120x5120 8.8 / 9.7 / 11.9 against 11.6 / 11.8 / 11.6,
// 4096x14336 12.7 / 15.1 / 18.5 against 16.0 / 16.4 / 16.3, 17408x5120 17.5 /
// 19.5 / 23.8 against 21.8 / 21.5 / 21.7.
struct PlainRows {
  const void* x;
  int64_t ldx;
  int32_t k;
};
constexpr int kFusedTokens = 3;

template <int BP, int WAVES, int XDT = 0>
__global__ __launch_bounds__(64 * WAVES) void k_f8_rows(PanelOperand W, PanelOperand X, PlainRows plain, F8Out out) {
  __shared__ f32x4_t part[WAVES][BP][64];
  // codes of the wavefront's four steps, [step][token][128], and exponent bytes
  __shared__ __attribute__((aligned(16))) char turn[XDT ? WAVES : 1][4 * kFusedTokens * 128];
  __shared__ uint32_t exps[XDT ? WAVES : 1][kFusedTokens];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t pw = int32_t(blockIdx.x), px = int32_t(blockIdx.y) * BP, steps = W.steps;
  const int64_t pitch = int64_t(steps) * kPanelStep;
  // One resource per panel, ending with it: steps behind the last are zeros.
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(W.data + pw * pitch, int32_t(pitch));
  __amdgpu_buffer_rsrc_t rx[BP];
#pragma unroll
  for (int j = 0; j < BP; ++j) {
    const bool ok = !XDT && (px + j) * 16 < X.rows16;
    rx[j] = make_rsrc(X.data + (ok ? px + j : 0) * pitch, ok ? int32_t(pitch) : 0);
  }
  f32x4_t acc[BP];
#pragma unroll
  for (int j = 0; j < BP; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int32_t s = wave * 4; s < steps; s += WAVES * 4) {
    u32x4_t a[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        a[t][h] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (s + t) * 2048 + h * 1024 + lane * 16, 0, HYB_W_AUX));
    const uint32_t sa = W.scale[int64_t(s >> 2) * W.scale_pitch + pw * 16 + (lane & 15)];
    if constexpr (XDT != 0) {
      // one wavefront writes and reads its own LDS: its accesses done suffices
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int r = 0; r < kFusedTokens; ++r) {
        if (r >= out.m) break;
        Eight<XDT> v = load8<XDT>(plain.x, r * plain.ldx, s * 128 + lane * 8, plain.k);
        trim8<XDT>(v, s * 128 + lane * 8, plain.k);
        uint32_t top = top_of<XDT>(v);
        const bool mark = __any(top >= kF32Inf);
        if (mark) top = top_finite<XDT>(v);
        const uint32_t e = s + (lane >> 4) < steps ? block_exponent(max16(top)) : 127u;
        *reinterpret_cast<uint2*>(turn[wave] + ((lane >> 4) * kFusedTokens + r) * 128 + (lane & 15) * 8) =
            codes8<XDT>(v, e, mark);
        const uint32_t word = __builtin_amdgcn_readlane(e, 0) | __builtin_amdgcn_readlane(e, 16) << 8 |
                              __builtin_amdgcn_readlane(e, 32) << 16 | __builtin_amdgcn_readlane(e, 48) << 24;
        if (lane == 0) exps[wave][r] = word;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int j = 0; j < BP; ++j) {
      const int32_t xr = (px + j) * 16 + (lane & 15);
      uint32_t sb;
      if constexpr (XDT != 0)
        sb = xr < out.m ? exps[wave][xr] : 127u;
      else
        sb = X.scale[int64_t(s >> 2) * X.scale_pitch + (xr < X.rows16 ? xr : 0)];
      auto step = [&](auto byte) {
        constexpr int t = decltype(byte)::value;
        u32x4_t b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (XDT != 0)
            b[h] = xr < out.m ? *reinterpret_cast<const u32x4_t*>(turn[wave] + (t * kFusedTokens + xr) * 128 + h * 64 +
                                                                  (lane >> 4) * 16)
                              : u32x4_t{0, 0, 0, 0};
          else
            b[h] = __builtin_bit_cast(
                u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx[j], (s + t) * 2048 + h * 1024 + lane * 16, 0, 0));
        }
        acc[j] = panel_mfma<kF8Wide, t>(panel_regs<kF8Wide, t>(a[t][0], a[t][1], sa),
                                        panel_regs<kF8Wide, t>(b[0], b[1], sb), acc[j], sa, sb);
      };
      step(std::integral_constant<int, 0>());
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 2>());
      step(std::integral_constant<int, 3>());
    }
  }
#pragma unroll
  for (int j = 0; j < BP; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  for (int t = threadIdx.x; t < BP * 64; t += 64 * WAVES) {
    const int j = t >> 6, l = t & 63;
    f32x4_t v = part[0][j][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const f32x4_t u = part[w][j][l];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    }
    f8_store4(out, int64_t(px + j) * 16 + (l & 15), pw * 16 + (l >> 4) * 4, v);
  }
}

// More tokens: AP x BP panels per workgroup through LDS, bound by the matrix
// instructions and, on a chip that lowers its clock under them, by power:
// 17408x5120 at 4096 tokens, bf16 to bf16, 322 us with the quantising (2.3
// PFLOP/s; the library's 8-bit product without block scales takes 330).  The
// first `whole`
// tiles (whole rounds of the compute units) run over all of k; each of the
// rest is cut into `parts`, whose sums are left in `ws` (wavefront by
// wavefront, as they lie in registers) for k_f8_sum.
template <int KIND, int AP, int BP, int WA, int WB, int STAGES>
__global__ __launch_bounds__(64 * WA * WB) void k_f8_tile(PanelOperand W, PanelOperand X, F8Out out,
                                                          int32_t whole, int parts, f32x4_t* __restrict__ ws) {
  typedef PanelTile<KIND, AP, BP, WA, WB, STAGES> T;
  extern __shared__ __attribute__((aligned(1024))) char f8_smem[];
  const int32_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  const int32_t id = int32_t(blockIdx.x), rest = id - whole;
  int32_t ab, bb, s0 = 0, s1 = W.steps;
  panel_block(rest < 0 ? panel_order(id, whole) : whole + rest / parts, na, nb, ab, bb);
  f32x4_t acc[T::kA][T::kB];
  if (rest >= 0) {
    const int32_t part = rest % parts, quads = (W.steps + 3) / 4;  // a part is a whole number of four steps
    s0 = int32_t(int64_t(quads) * part / parts) * 4;
    if (part + 1 < parts) s1 = int32_t(int64_t(quads) * (part + 1) / parts) * 4;
  }
  T::run(W, X, ab * AP, bb * BP, s0, s1, f8_smem, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave % WA, wb = wave / WA;
  if (rest >= 0) {
    f32x4_t* p = ws + int64_t(rest) * (AP * BP * 64) + wave * (T::kA * T::kB * 64) + lane;
#pragma unroll
    for (int j = 0; j < T::kB; ++j)
#pragma unroll
      for (int i = 0; i < T::kA; ++i) p[(i * T::kB + j) * 64] = acc[i][j];
    return;
  }
  if (out.ydt != HYB_F32) {
    __syncthreads();  // the tile's LDS stages are free
    const int64_t m0 = int64_t(bb * BP + wb * T::kB) * 16;
    const int32_t n0 = (ab * AP + wa * T::kA) * 16;
    panel_rows16<T::kA, T::kB>(
        f8_smem + wave * (T::kA * T::kB * 512), lane, lane & 15,
        [&](int i, int j) {
          const f32x4_t v = acc[i][j];
          return out.ydt == HYB_BF16 ? round16x4<HYB_BF16>(v[0], v[1], v[2], v[3])
                                     : round16x4<HYB_F16>(v[0], v[1], v[2], v[3]);
        },
        [&](int row, int col, uint4 u) {
          const int64_t m = m0 + row;
          const int32_t n = n0 + col;
          if (m >= out.m || n >= out.n) return;
          uint16_t* p = static_cast<uint16_t*>(out.y) + m * out.ldy + n;
          if (n + 8 <= out.n) {
            *reinterpret_cast<Bytes16*>(p) = Bytes16{{u.x, u.y, u.z, u.w}};
          } else {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (n + e < out.n) p[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
          }
        });
    return;
  }
#pragma unroll
  for (int j = 0; j < T::kB; ++j)
#pragma unroll
    for (int i = 0; i < T::kA; ++i)
      f8_store4(out, int64_t(bb * BP + wb * T::kB + j) * 16 + (lane & 15),
                (ab * AP + wa * T::kA + i) * 16 + (lane >> 4) * 4, acc[i][j]);
}

// Adds the parts of a tile in order and stores the outputs: one workgroup per
// four of a tile's AP x BP panel products.  Bound by memory (17408x5120 at 256
// tokens 4 us).
template <int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(256) void k_f8_sum(const f32x4_t* __restrict__ ws, int32_t na, int32_t nb, int32_t whole,
                                                int parts, F8Out out) {
  constexpr int kA = AP / WA, kB = BP / WB;
  const int lane = threadIdx.x & 63;
  const int c = int(blockIdx.y) * 4 + (threadIdx.x >> 6);  // wavefront, i, j of the tile
  const int wave = c / (kA * kB), i = c % (kA * kB) / kB, j = c % kB;
  int32_t ab, bb;
  panel_block(whole + int32_t(blockIdx.x), na, nb, ab, bb);
  const f32x4_t* p = ws + int64_t(blockIdx.x) * parts * (AP * BP * 64) + c * 64 + lane;
  f32x4_t v = p[0];
  for (int t = 1; t < parts; ++t) {
    const f32x4_t u = p[int64_t(t) * (AP * BP * 64)];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += u[e];
  }
  f8_store4(out, int64_t(bb * BP + wave / WA * kB + j) * 16 + (lane & 15),
            (ab * AP + wave % WA * kA + i) * 16 + (lane >> 4) * 4, v);
}

// Zeros (k = 0).
__global__ __launch_bounds__(256) void k_f8_zero(F8Out o) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < int64_t(o.n) * o.m; i += int64_t(gridDim.x) * 256)
    store_out(o.y, o.ydt, i / o.n * o.ldy + i % o.n, 0.f);
}

template <int KIND, int AP, int BP, int WA, int WB, int STAGES>
hipError_t launch_tile(const PanelOperand& W, const PanelOperand& X, const F8Out& o, const F8Route& r, float* ws,
                       hipStream_t s) {
  typedef PanelTile<KIND, AP, BP, WA, WB, STAGES> T;
  const void* fn = reinterpret_cast<const void*>(&k_f8_tile<KIND, AP, BP, WA, WB, STAGES>);
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
  if (e != hipSuccess) return e;
  const int64_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  const int64_t whole = ws && r.parts > 1 ? r.whole : na * nb, rest = na * nb - whole;
  f32x4_t* sums = reinterpret_cast<f32x4_t*>(ws);
  hipLaunchKernelGGL((k_f8_tile<KIND, AP, BP, WA, WB, STAGES>), dim3(unsigned(whole + rest * r.parts)),
                     dim3(64 * WA * WB), T::kLds, s, W, X, o, int32_t(whole), r.parts, sums);
  if (rest > 0)
    hipLaunchKernelGGL((k_f8_sum<AP, BP, WA, WB>), dim3(unsigned(rest), AP * BP / 4), dim3(256), 0, s, sums,
                       int32_t(na), int32_t(nb), int32_t(whole), r.parts, o);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_route(const F8Route& r, const PanelOperand& W, const PanelOperand& X, const F8Out& o, float* ws,
                        hipStream_t s) {
  if (r.ap == 16 && r.bp == 16) return launch_tile<KIND, 16, 16, 2, 4, 2>(W, X, o, r, ws, s);
  if (r.ap == 16) return launch_tile<KIND, 16, 8, 4, 2, 2>(W, X, o, r, ws, s);
  return launch_tile<KIND, 8, 8, 2, 4, 4>(W, X, o, r, ws, s);
}

template <int XDT>
void launch_fused(const PanelOperand& W, const PlainRows& x, const F8Out& o, hipStream_t s) {
  hipLaunchKernelGGL((k_f8_rows<1, 8, XDT>), dim3(unsigned(W.rows16 / 16)), dim3(512), 0, s, W, PanelOperand{}, x, o);
}

}  // namespace

bool f8_fused(int64_t n, int64_t k, int64_t m, int y_dtype) {
  if (m > kFusedTokens || k == 0) return false;
  const F8Route r = f8_route(n, k, m, y_dtype == HYB_F32, device_cus());
  return r.waves == 8 && r.bp == 1;
}

hipError_t launch_f8_fused(const hyb_f8& w, int64_t n, int64_t k, const void* x, int x_dtype, int64_t m, int64_t ldx,
                           void* y, int y_dtype, int64_t ldy, hipStream_t s) {
  const PanelOperand W{static_cast<const char*>(w.codes), int32_t(f8_rows16(n)), int32_t(f8_steps(k)),
                       static_cast<const uint32_t*>(w.scales), f8_rows16(n)};
  const F8Out o{y, ldy, int32_t(n), int32_t(m), y_dtype};
  const PlainRows p{x, ldx, int32_t(k)};
  if (x_dtype == HYB_F32)
    launch_fused<HYB_F32>(W, p, o, s);
  else if (x_dtype == HYB_BF16)
    launch_fused<HYB_BF16>(W, p, o, s);
  else
    launch_fused<HYB_F16>(W, p, o, s);
  return hipGetLastError();
}

hipError_t launch_f8_quantize(const void* a, int dtype, int64_t rows, int64_t k, int64_t lda, int kind,
                              const hyb_f8& dst, hipStream_t s) {
  const int32_t panels = int32_t(f8_rows16(rows) / 16), steps = int32_t(f8_steps(k));
  const unsigned quads = unsigned((steps + 3) / 4);
  // workgroups along a panel's steps (its bytes of scales beyond the last step
  // are written too), and in all
  const int32_t across = int32_t(kind == HYB_F8_WEIGHT ? quads * 4 : quads);
  const int64_t grid = int64_t(kind == HYB_F8_WEIGHT ? (panels + 7) / 8 : panels) * across;
  // (2^37 elements: more than a card holds)
  if (grid * (kind == HYB_F8_WEIGHT ? 512 : 256) >= int64_t(1) << 32) return hipErrorInvalidValue;
  char* codes = static_cast<char*>(dst.codes);
  char* scales = static_cast<char*>(dst.scales);
#define HYB_F8_QUANT(DT)                                                                                             \
  if (kind == HYB_F8_WEIGHT)                                                                                         \
    hipLaunchKernelGGL((k_f8_quantize<DT, true>), dim3(unsigned(grid)), dim3(512), 0, s, a, rows, int32_t(k), lda, codes,            \
                       scales, panels, steps, across);                                                               \
  else                                                                                                               \
    hipLaunchKernelGGL((k_f8_quantize<DT, false>), dim3(unsigned(grid)), dim3(256), 0, s, a, rows, int32_t(k), lda, codes,           \
                       scales, panels, steps, across)
  if (dtype == HYB_F32) {
    HYB_F8_QUANT(HYB_F32);
  } else if (dtype == HYB_BF16) {
    HYB_F8_QUANT(HYB_BF16);
  } else {
    HYB_F8_QUANT(HYB_F16);
  }
#undef HYB_F8_QUANT
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const hyb_f8& src, int64_t rows, int64_t k, void* a, int dtype, int64_t lda,
                                hipStream_t s) {
  const int32_t panels = int32_t(f8_rows16(rows) / 16), steps = int32_t(f8_steps(k));
  const dim3 grid(unsigned(panels), unsigned((steps + 3) / 4));
  const char* codes = static_cast<const char*>(src.codes);
  const uint32_t* scales = static_cast<const uint32_t*>(src.scales);
  if (dtype == HYB_F32)
    hipLaunchKernelGGL((k_f8_dequantize<HYB_F32>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda, a,
                       panels, steps);
  else if (dtype == HYB_BF16)
    hipLaunchKernelGGL((k_f8_dequantize<HYB_BF16>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda,
                       a, panels, steps);
  else
    hipLaunchKernelGGL((k_f8_dequantize<HYB_F16>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda, a,
                       panels, steps);
  return hipGetLastError();
}

hipError_t launch_f8_gemm(const hyb_f8& w, int64_t n, int64_t k, const hyb_f8& x, int64_t m, void* y, int y_dtype,
                          int64_t ldy, float* ws, hipStream_t s, int64_t w_pitch) {
  const F8Out o{y, ldy, int32_t(n), int32_t(m), y_dtype};
  if (k == 0) {
    const int64_t blocks = (n * m + 255) / 256;
    hipLaunchKernelGGL(k_f8_zero, dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, o);
    return hipGetLastError();
  }
  const int32_t steps = int32_t(f8_steps(k));
  const PanelOperand W{static_cast<const char*>(w.codes), int32_t(f8_rows16(n)), steps,
                       static_cast<const uint32_t*>(w.scales), w_pitch ? w_pitch : f8_rows16(n)};
  const PanelOperand X{static_cast<const char*>(x.codes), int32_t(f8_rows16(m)), steps,
                       static_cast<const uint32_t*>(x.scales), f8_rows16(m)};
  const F8Route r = f8_route(n, k, m, y_dtype == HYB_F32, device_cus());
  if (r.waves) {
    const dim3 grid(unsigned(W.rows16 / 16), unsigned((X.rows16 / 16 + r.bp - 1) / r.bp));
    if (r.bp == 1)
      hipLaunchKernelGGL((k_f8_rows<1, 8>), grid, dim3(512), 0, s, W, X, PlainRows{}, o);
    else if (r.bp == 2)
      hipLaunchKernelGGL((k_f8_rows<2, 8>), grid, dim3(512), 0, s, W, X, PlainRows{}, o);
    else
      hipLaunchKernelGGL((k_f8_rows<4, 8>), grid, dim3(512), 0, s, W, X, PlainRows{}, o);
    return hipGetLastError();
  }
  return y_dtype == HYB_F32 ? launch_route<kF8Wide>(r, W, X, o, ws, s) : launch_route<kF8>(r, W, X, o, ws, s);
}

}  // namespace hyb
