// Kernels of the 8-bit block-scaled matrices (include/hyb_f8.h): quantise,
// read back, and the product on the scaled matrix instructions.
#include <type_traits>

#include "hyb_f8_internal.h"
#include "hyb_panel.h"

namespace hyb {
namespace {

// ------------------------------------------------------ quantise, read back --

// 16 columns c0.. of one row as fp32; zeros behind the row's end.  `vec`:
// every row starts 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load16(const void* a, int64_t base, int32_t c0, int32_t k, bool row_ok, bool vec,
                                       float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  if (!row_ok || c0 >= k) return;
  if (vec && c0 + 16 <= k) {
    if constexpr (DT == HYB_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a) + base + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = p[i];
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a) + base + c0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = p[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = widen16<DT>(w[j] & 0xFFFFu);
          v[8 * i + 2 * j + 1] = widen16<DT>(w[j] >> 16);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (c0 + i < k) {
      if constexpr (DT == HYB_F32)
        v[i] = static_cast<const float*>(a)[base + c0 + i];
      else
        v[i] = widen16<DT>(static_cast<const uint16_t*>(a)[base + c0 + i]);
    }
  }
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

constexpr uint32_t kF32Inf = 0x7F800000u;

// Magnitude bits of the largest finite element.
__device__ __forceinline__ uint32_t top_finite(const float (&v)[16], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
    top = u < kF32Inf && u > top ? u : top;
  }
  return top;
}

// 16 codes of elements already divided by the scale (|.| <= 448, or not
// finite: made NaN first, the conversion leaves NaN as the NaN code).
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = v[4 * i + j];
      const bool finite = (__builtin_bit_cast(uint32_t, a) & 0x7FFFFFFFu) < kF32Inf;
      f[j] = finite ? a * inv : __builtin_nanf("");
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    w[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One wavefront per panel and four steps (512 columns): lane L holds, of each
// step, its row's columns 16 (L/16) + 0..15 of both halves, so the codes
// leave as 1 KiB stores in panel order and a row's maximum needs the four
// lanes of that row.  A weight block is eight panels: a workgroup of eight
// wavefronts, whose maxima meet in LDS.  Bound by memory (one read of the
// matrix, half or a quarter as many bytes written).
template <int DT, bool WEIGHT>
__global__ __launch_bounds__(512) void k_f8_quantize(const void* __restrict__ a, int64_t rows, int32_t k, int64_t lda,
                                                     int vec, char* __restrict__ codes, uint32_t* __restrict__ scales,
                                                     int32_t panels, int32_t steps) {
  __shared__ uint32_t top_lds[8][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4;
  const int64_t panel = int64_t(blockIdx.x) * 8 + wave;
  const int32_t s0 = int32_t(blockIdx.y) * 4;
  const int64_t row = panel * 16 + (lane & 15);
  const bool live = panel < panels;
  const int64_t base = row * lda;
  float v[4][2][16];
  uint32_t top[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load16<DT>(a, base, (s0 + s) * 128 + h * 64 + q * 16, k, row < rows, vec, v[s][h]);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t t = top_finite(v[s][0], 0u);
    t = top_finite(v[s][1], t);
    uint32_t o = __shfl_xor(t, 16);
    t = o > t ? o : t;
    o = __shfl_xor(t, 32);
    top[s] = o > t ? o : t;
  }
  if constexpr (WEIGHT) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int d = 1; d < 16; d *= 2) {
        const uint32_t o = __shfl_xor(top[s], d);
        top[s] = o > top[s] ? o : top[s];
      }
      if (lane == 0) top_lds[wave][s] = top[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int w = 0; w < 8; ++w) top[s] = top_lds[w][s] > top[s] ? top_lds[w][s] : top[s];
  }
  if (!live) return;
  uint32_t word = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t e = s0 + s < steps ? block_exponent(top[s]) : 127u;
    word |= e << (8 * s);
    if (s0 + s >= steps) continue;
    const float inv = exp2_byte(254u - e);
    char* dst = codes + (panel * steps + s0 + s) * kPanelStep + lane * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + h * 1024) = codes16(v[s][h], inv);
  }
  if (q == 0) scales[int64_t(s0 / 4) * panels * 16 + row] = row < rows ? word : 0x7F7F7F7Fu;
}

template <int DT>
__global__ __launch_bounds__(256) void k_f8_dequantize(const char* __restrict__ codes,
                                                       const uint32_t* __restrict__ scales, int64_t rows, int32_t k,
                                                       int64_t lda, int vec, void* __restrict__ a, int32_t panels,
                                                       int32_t steps) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = int64_t(blockIdx.x) * 4 + wave;
  const int64_t row = panel * 16 + (lane & 15);
  if (panel >= panels || row >= rows) return;
  const int32_t s0 = int32_t(blockIdx.y) * 4;
  const uint32_t word = scales[int64_t(s0 / 4) * panels * 16 + row];
  for (int s = 0; s < 4 && s0 + s < steps; ++s) {
    const float scale = exp2_byte((word >> (8 * s)) & 0xFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = *reinterpret_cast<const uint4*>(codes + (panel * steps + s0 + s) * kPanelStep + h * 1024 + lane * 16);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float f[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[4 * i] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 0) * scale;
        f[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 1) * scale;
        f[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 2) * scale;
        f[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(int(w[i]), 3) * scale;
      }
      const int32_t c0 = (s0 + s) * 128 + h * 64 + (lane >> 4) * 16;
      if (c0 >= k) continue;
      const int64_t at = row * lda + c0;
      if (vec && c0 + 16 <= k) {
        if constexpr (DT == HYB_F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(static_cast<float*>(a) + at)[i] =
                make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = round16<DT>(f[2 * i]) | uint32_t(round16<DT>(f[2 * i + 1])) << 16;
          uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a) + at);
          p[0] = make_uint4(o[0], o[1], o[2], o[3]);
          p[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c0 + i < k) store_out(a, DT, at + i, f[i]);
      }
    }
  }
}

// ------------------------------------------------------------------ product --

struct F8Out {
  void* y;
  int64_t ldy;
  int32_t n, m, ydt, vec;  // vec: four-element stores are aligned
};

// Four outputs n..n+3 of token m.
__device__ __forceinline__ void f8_store4(const F8Out& o, int64_t m, int32_t n, f32x4_t v) {
  if (m >= o.m || n >= o.n) return;
  const int64_t at = m * o.ldy + n;
  if (o.vec && n + 4 <= o.n) {
    if (o.ydt == HYB_F32) {
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(o.y) + at) = v;
    } else {
      uint16_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = o.ydt == HYB_BF16 ? round16<HYB_BF16>(v[e]) : round16<HYB_F16>(v[e]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.y) + at) =
          make_uint2(h[0] | uint32_t(h[1]) << 16, h[2] | uint32_t(h[3]) << 16);
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
// kind costs nothing here and serves every output type.
template <int BP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_f8_rows(PanelOperand W, PanelOperand X, F8Out out) {
  __shared__ f32x4_t part[WAVES][BP][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t pw = int32_t(blockIdx.x), px = int32_t(blockIdx.y) * BP, steps = W.steps;
  const int64_t pitch = int64_t(steps) * kPanelStep;
  // One resource per panel, ending with it: steps behind the last are zeros.
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(W.data + pw * pitch, int32_t(pitch));
  __amdgpu_buffer_rsrc_t rx[BP];
#pragma unroll
  for (int j = 0; j < BP; ++j) {
    const bool ok = (px + j) * 16 < X.rows16;
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
#pragma unroll
    for (int j = 0; j < BP; ++j) {
      const int32_t xr = (px + j) * 16 + (lane & 15);
      const uint32_t sb = X.scale[int64_t(s >> 2) * X.scale_pitch + (xr < X.rows16 ? xr : 0)];
      auto step = [&](auto byte) {
        constexpr int t = decltype(byte)::value;
        u32x4_t b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b[h] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx[j], (s + t) * 2048 + h * 1024 + lane * 16, 0, 0));
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

template <int KIND, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void k_f8_tile(PanelOperand W, PanelOperand X, F8Out out) {
  typedef PanelTile<KIND, AP, BP, WA, WB> T;
  extern __shared__ __attribute__((aligned(1024))) char f8_smem[];
  const int32_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  int32_t ab, bb;
  panel_block(int32_t(blockIdx.x), na * nb, na, nb, ab, bb);
  f32x4_t acc[T::kA][T::kB];
  T::run(W, X, ab * AP, bb * BP, 0, W.steps, f8_smem, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wa = wave % WA, wb = wave / WA;
#pragma unroll
  for (int j = 0; j < T::kB; ++j)
#pragma unroll
    for (int i = 0; i < T::kA; ++i)
      f8_store4(out, int64_t(bb * BP + wb * T::kB + j) * 16 + (lane & 15),
                (ab * AP + wa * T::kA + i) * 16 + (lane >> 4) * 4, acc[i][j]);
}

// Zeros (k = 0).
__global__ __launch_bounds__(256) void k_f8_zero(F8Out o) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < int64_t(o.n) * o.m) store_out(o.y, o.ydt, i / o.n * o.ldy + i % o.n, 0.f);
}

template <int KIND, int AP, int BP, int WA, int WB>
hipError_t launch_tile(const PanelOperand& W, const PanelOperand& X, const F8Out& o, hipStream_t s) {
  typedef PanelTile<KIND, AP, BP, WA, WB> T;
  const void* fn = reinterpret_cast<const void*>(&k_f8_tile<KIND, AP, BP, WA, WB>);
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
  if (e != hipSuccess) return e;
  const int64_t na = (W.rows16 + 16 * AP - 1) / (16 * AP), nb = (X.rows16 + 16 * BP - 1) / (16 * BP);
  hipLaunchKernelGGL((k_f8_tile<KIND, AP, BP, WA, WB>), dim3(unsigned(na * nb)), dim3(64 * WA * WB), T::kLds, s, W, X, o);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const void* a, int dtype, int64_t rows, int64_t k, int64_t lda, int kind,
                              const hyb_f8& dst, hipStream_t s) {
  const int32_t panels = int32_t(f8_rows16(rows) / 16), steps = int32_t(f8_steps(k));
  const int esize = dtype == HYB_F32 ? 4 : 2;
  const int vec = reinterpret_cast<uintptr_t>(a) % 16 == 0 && lda * esize % 16 == 0;
  const dim3 grid(unsigned((panels + 7) / 8), unsigned((steps + 3) / 4));
  char* codes = static_cast<char*>(dst.codes);
  uint32_t* scales = static_cast<uint32_t*>(dst.scales);
#define HYB_F8_QUANT(DT)                                                                                             \
  if (kind == HYB_F8_WEIGHT)                                                                                         \
    hipLaunchKernelGGL((k_f8_quantize<DT, true>), grid, dim3(512), 0, s, a, rows, int32_t(k), lda, vec, codes,       \
                       scales, panels, steps);                                                                       \
  else                                                                                                               \
    hipLaunchKernelGGL((k_f8_quantize<DT, false>), grid, dim3(512), 0, s, a, rows, int32_t(k), lda, vec, codes,      \
                       scales, panels, steps)
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
  const int esize = dtype == HYB_F32 ? 4 : 2;
  const int vec = reinterpret_cast<uintptr_t>(a) % 16 == 0 && lda * esize % 16 == 0;
  const dim3 grid(unsigned((panels + 3) / 4), unsigned((steps + 3) / 4));
  const char* codes = static_cast<const char*>(src.codes);
  const uint32_t* scales = static_cast<const uint32_t*>(src.scales);
  if (dtype == HYB_F32)
    hipLaunchKernelGGL((k_f8_dequantize<HYB_F32>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda, vec, a,
                       panels, steps);
  else if (dtype == HYB_BF16)
    hipLaunchKernelGGL((k_f8_dequantize<HYB_BF16>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda, vec,
                       a, panels, steps);
  else
    hipLaunchKernelGGL((k_f8_dequantize<HYB_F16>), grid, dim3(256), 0, s, codes, scales, rows, int32_t(k), lda, vec, a,
                       panels, steps);
  return hipGetLastError();
}

hipError_t launch_f8_gemm(const hyb_f8& w, int64_t n, int64_t k, const hyb_f8& x, int64_t m, void* y, int y_dtype,
                          int64_t ldy, float* ws, hipStream_t s) {
  const int esize = y_dtype == HYB_F32 ? 4 : 2;
  const F8Out o{y,      ldy, int32_t(n), int32_t(m), y_dtype,
                reinterpret_cast<uintptr_t>(y) % (4 * esize) == 0 && ldy % 4 == 0};
  if (k == 0) {
    hipLaunchKernelGGL(k_f8_zero, dim3(unsigned((n * m + 255) / 256)), dim3(256), 0, s, o);
    return hipGetLastError();
  }
  const int32_t steps = int32_t(f8_steps(k));
  const PanelOperand W{static_cast<const char*>(w.codes), int32_t(f8_rows16(n)), steps,
                       static_cast<const uint32_t*>(w.scales), f8_rows16(n)};
  const PanelOperand X{static_cast<const char*>(x.codes), int32_t(f8_rows16(m)), steps,
                       static_cast<const uint32_t*>(x.scales), f8_rows16(m)};
  const F8Route r = f8_route(n, k, m, device_cus());
  (void)ws;
  if (r.waves) {
    const dim3 grid(unsigned(W.rows16 / 16), unsigned((X.rows16 / 16 + r.bp - 1) / r.bp));
    if (r.bp == 1)
      hipLaunchKernelGGL((k_f8_rows<1, 8>), grid, dim3(512), 0, s, W, X, o);
    else if (r.bp == 2)
      hipLaunchKernelGGL((k_f8_rows<2, 8>), grid, dim3(512), 0, s, W, X, o);
    else
      hipLaunchKernelGGL((k_f8_rows<4, 8>), grid, dim3(512), 0, s, W, X, o);
    return hipGetLastError();
  }
  const bool wide = y_dtype == HYB_F32;  // kF8Wide
  if (r.ap == 16)
    return wide ? launch_tile<kF8Wide, 16, 16, 2, 4>(W, X, o, s) : launch_tile<kF8, 16, 16, 2, 4>(W, X, o, s);
  return wide ? launch_tile<kF8Wide, 8, 8, 2, 2>(W, X, o, s) : launch_tile<kF8, 8, 8, 2, 2>(W, X, o, s);
}

}  // namespace hyb
