// Kernels of the 4-bit weights (include/hyb_q4.h): quantise, read back, the
// product, and the gated product of two weights (include/hyb_gated.h).
#include <type_traits>

#include "hyb_act.h"
#include "hyb_panel.h"
#include "hyb_q4_internal.h"
#include "hyb_stream.h"

namespace hyb {
namespace {

// ------------------------------------------------------ quantise, read back --

// Eight columns of one row, as loaded: two elements to a word, or one for fp32.
template <int DT>
struct Eight4 {
  uint32_t w[DT == HYB_F32 ? 8 : 4];
};

// Columns c0.. of the row at element `base`.  A lane at or behind the row's end
// loads the row's last eight columns (k >= 8), so that a wavefront's loads need no
// branches and are all under way at once; trim4 then moves its columns into place
// and zeros the rest.
template <int DT>
__device__ __forceinline__ Eight4<DT> load4(const void* a, int64_t base, int32_t c0, int32_t k) {
  Eight4<DT> r;
  constexpr int kWords = DT == HYB_F32 ? 8 : 4;
  if (k < 8) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = 0;
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
    const Bytes16 u = stream_load(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[4 * i + j] = u.w[j];
  }
  return r;
}

// Eight 16-bit columns moved down by `by` (none if it is not positive), zeros
// behind.
__device__ __forceinline__ uint4 move_down(uint4 u, int by) {
  if (by >= 8) return make_uint4(0, 0, 0, 0);
  if (by > 0) {
    if (by & 4) u = make_uint4(u.z, u.w, 0, 0);
    if (by & 2) u = make_uint4(u.y, u.z, u.w, 0);
    if (by & 1)
      u = make_uint4(u.x >> 16 | u.y << 16, u.y >> 16 | u.z << 16, u.z >> 16 | u.w << 16, u.w >> 16);
  }
  return u;
}

template <int DT>
__device__ __forceinline__ void trim4(Eight4<DT>& r, int32_t c0, int32_t k) {
  if (k < 8) return;
  const int32_t by = c0 - (k - 8);
  if constexpr (DT == HYB_F32) {
#pragma unroll
    for (int d = 1; d < 8; d *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (by > 0 && (by & d)) r.w[i] = i + d < 8 ? r.w[i + d < 8 ? i + d : 0] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = by >= 8 ? 0 : r.w[i];
  } else {
    const uint4 u = move_down(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), by);
    r.w[0] = u.x;
    r.w[1] = u.y;
    r.w[2] = u.z;
    r.w[3] = u.w;
  }
}

// Scale byte of a group from its largest magnitude's bits: e + 127 with the
// smallest e in [-125, 125] for which the magnitude is at most 7 * 2^e (7 is
// 1.75 * 2^2); 127 for zero, 255 for infinities and NaN.
__device__ __forceinline__ uint32_t group_byte(uint32_t top) {
  if (top == 0) return 127u;
  if (top >= 0x7F800000u) return 255u;
  const int e = int((top + 0x1FFFFFu) >> 23) - 2;  // the next binade from above 1.75 on
  return uint32_t(e < 2 ? 2 : e > 252 ? 252 : e);
}

// One workgroup per panel, a wavefront per 512 columns at a time: a load covers
// them in one row (8 columns per lane, four lanes to a group), codes and scales are
// put into the stream's order in LDS.  Bound by memory: 28672x8192 bf16, 470 MB read
// and 125 MB written, 111-128 us (4.6-5.4 TB/s; with loads that the caches keep 166, and
// so with 128 columns of four rows to a load 186).
template <int DT>
__global__ __launch_bounds__(256) void k_q4_quantize(const void* __restrict__ a, int64_t n, int32_t k, int64_t lda,
                                                     int32_t steps, int64_t rows16, char* __restrict__ codes,
                                                     char* __restrict__ scales) {
  // units and steps 4 and 16 banks apart: a row's 64 words lie on 64 banks
  constexpr int kUnit = 256 + 16, kStep = 4 * kUnit;
  constexpr int kRows = DT == HYB_F32 ? 4 : 8;  // loaded at once
  __shared__ __attribute__((aligned(16))) char stage[4][4 * kStep + 256];
  __shared__ uint32_t tops[4][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = blockIdx.x;
  const int32_t quads = (steps + 3) / 4;
  const int live = n - panel * 16 < 16 ? int(n - panel * 16) : 16;  // rows
  const int j = lane & 15;
  char* mine = stage[wave];
  char* at = mine + (lane >> 4) * kStep + (j & 3) * kUnit + (j >> 2) * 4;
  uint32_t best[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) best[r] = 0;
  // two sets of registers take turns, so that loads are under way during the
  // arithmetic
  Eight4<DT> regs[2][kRows];
  auto load = [&](Eight4<DT> (&in)[kRows], int32_t q, int r0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      in[r] = load4<DT>(a, (panel * 16 + (r0 + r < live ? r0 + r : live - 1)) * lda, q * 512 + lane * 8, k);
  };
  if (wave < quads) load(regs[0], wave, 0);
  for (int32_t q = wave; q < quads; q += 4) {
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += kRows) {
      Eight4<DT> (&in)[kRows] = regs[r0 / kRows & 1];
      if (r0 + kRows < 16)
        load(regs[(r0 / kRows + 1) & 1], q, r0 + kRows);
      else if (q + 4 < quads)
        load(regs[(r0 / kRows + 1) & 1], q + 4, 0);
      if ((q + 1) * 512 > k) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) trim4<DT>(in[r], q * 512 + lane * 8, k);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = in[r].w[DT == HYB_F32 ? e : e / 2];
          v[e] = DT == HYB_F32 ? __builtin_bit_cast(float, w)
                               : widen16<DT == HYB_F32 ? HYB_BF16 : DT>(e & 1 ? w >> 16 : w & 0xFFFFu);
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = v[e];
          const uint32_t b = __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
          top = b > top ? b : top;
        }
        // over the four lanes of the group
        uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(top), 0xB1, 0xF, 0xF, true));
        top = o > top ? o : top;
        o = uint32_t(__builtin_amdgcn_update_dpp(0, int(top), 0x4E, 0xF, 0xF, true));
        top = r0 + r < live ? (o > top ? o : top) : 0;
        const uint32_t byte = group_byte(top);
        const float scale = __builtin_bit_cast(float, byte << 23);
        uint32_t code = 0;
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0], v[1], scale, 0);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2], v[3], scale, 1);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4], v[5], scale, 2);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6], v[7], scale, 3);
        code = r0 + r < live && byte != 255u ? code : 0;
        *reinterpret_cast<uint32_t*>(at + (r0 + r) * 16) = code;
        if ((j & 3) == 0) mine[4 * kStep + (r0 + r) * 16 + (lane >> 2)] = char(byte);
        if (byte != 255u && top != 0 && byte > best[r0 + r]) best[r0 + r] = byte;
      }
    }
    // one wavefront writes and reads its own part: its accesses done suffices
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (q * 4 + s < steps)
        *reinterpret_cast<uint4*>(codes + (panel * steps + q * 4 + s) * kQ4StepBytes + lane * 16) =
            *reinterpret_cast<const uint4*>(mine + s * kStep + (lane >> 4) * kUnit + j * 16);
    *reinterpret_cast<uint32_t*>(scales + (q * rows16 + panel * 16) * 16 + lane * 4) =
        *reinterpret_cast<const uint32_t*>(mine + 4 * kStep + lane * 4);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    uint32_t b = best[r];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_xor(b, d);
      b = o > b ? o : b;
    }
    if (lane == 0) tops[wave][r] = b;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    uint32_t b = 0;
    for (int w = 0; w < 4; ++w) b = tops[w][threadIdx.x] > b ? tops[w][threadIdx.x] : b;
    scales[quads * rows16 * 16 + panel * 16 + threadIdx.x] = char(b == 0 ? 127u : b);
  }
}

// One wavefront per panel and step: codes through LDS into rows, 8 columns per
// lane.  Bound by memory: 28672x8192 to bf16, 595 MB, 94 us (6.3 TB/s; with stores that
// the caches keep 111, and the quantising of the next weight 128 instead of 111).  To
// fp32, whose 32 bytes a lane leave in two stores, the caches put the halves together:
// 277 us (3.8 TB/s; around them 491).
template <int DT, bool STREAM>
__global__ __launch_bounds__(256) void k_q4_dequantize(const char* __restrict__ codes,
                                                       const char* __restrict__ scales, int64_t n, int32_t k,
                                                       int64_t lda, int32_t steps, int64_t rows16,
                                                       void* __restrict__ a) {
  __shared__ __attribute__((aligned(16))) char stage[4][1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = blockIdx.x;
  const int32_t s = int32_t(blockIdx.y) * 4 + wave;
  if (s >= steps) return;
  char* mine = stage[wave];
  *reinterpret_cast<uint4*>(mine + lane * 16) =
      *reinterpret_cast<const uint4*>(codes + (panel * steps + s) * kQ4StepBytes + lane * 16);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int j = lane & 15, rr = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + rr;
    const int64_t row = panel * 16 + r;
    const int32_t c0 = s * 128 + j * 8;
    if (row >= n || c0 >= k) continue;
    const uint32_t code = *reinterpret_cast<const uint32_t*>(mine + (j & 3) * 256 + r * 16 + (j >> 2) * 4);
    const uint32_t byte = uint8_t(scales[((s >> 2) * rows16 + row) * 16 + (s & 3) * 4 + (j >> 2)]);
    const float scale = __builtin_bit_cast(float, byte << 23);
    float v[8];
    auto two = [&](auto sel) {
      constexpr int b = decltype(sel)::value;
      const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, scale, b);
      v[2 * b] = p[0];
      v[2 * b + 1] = p[1];
    };
    two(std::integral_constant<int, 0>());
    two(std::integral_constant<int, 1>());
    two(std::integral_constant<int, 2>());
    two(std::integral_constant<int, 3>());
    if constexpr (DT == HYB_F32) {
      float* p = static_cast<float*>(a) + row * lda + c0;
      if (c0 + 8 <= k) {
        Bytes16 u[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e >> 2].w[e & 3] = __builtin_bit_cast(uint32_t, v[e]);
        reinterpret_cast<Bytes16*>(p)[0] = u[0];
        reinterpret_cast<Bytes16*>(p)[1] = u[1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + e < k) p[e] = v[e];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(a) + row * lda + c0;
      if (c0 + 8 <= k) {
        Bytes16 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u.w[e] = round16x2<DT>(v[2 * e], v[2 * e + 1]);
        if constexpr (STREAM)
          stream_store(p, u);
        else
          *reinterpret_cast<Bytes16*>(p) = u;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + e < k) p[e] = round16<DT>(v[e]);
      }
    }
  }
}

// ----------------------------------------------------------------- products --

struct Q4Weight {
  const char* codes;
  const char* scales;
  const uint8_t* tops;
};

struct Q4Args {
  Q4Weight w[2];  // the second for the gated product
  int64_t rows16;
  int32_t steps, n, k;
  const uint16_t* x;
  int64_t ldx, m;
  void* y;
  int64_t ldy;
  int ydt, act;
  const char* xt;  // tiles: the activations as panels, of x_panel bytes
  int64_t x_panel;
  int32_t steps64;
  // tiles that run over all of k, and the parts each of the others is cut into,
  // whose sums are left in `ws`
  f32x4_t* ws;
  int32_t whole, parts;
};

// fp16 operands carry a row's values divided by 2^(top - 140): at most 6 * 2^13 (below
// fp16's 65504), and 2^-24, its smallest number, for half of a scale of 2^-36 of the
// row's largest.
constexpr int kTopLift = 140;

// The scale of group h of a word's four: its byte as the exponent of a float.
// (The conversion reads only the exponent: bits of the bytes around it may lie
// in the sign and the mantissa.)  For fp16 `lift` is kTopLift - top; the byte of a
// group of zeros may lie far above top, and stays short of 255, a NaN.
template <int DT>
__device__ __forceinline__ float group_scale(uint32_t word, int h, int lift) {
  if constexpr (DT == HYB_BF16) {
    return __builtin_bit_cast(float, h < 3 ? word << (23 - 8 * h) : word >> 1);
  } else {
    const int b = (word >> (8 * h)) & 0xFFu;
    const int e = b + lift < 0 ? 0 : b + lift > 254 ? 254 : b + lift;
    return __builtin_bit_cast(float, uint32_t(b == 255 ? 255 : e) << 23);
  }
}

// Eight codes as an operand of the 16-bit matrix instruction.
template <int DT>
__device__ __forceinline__ uint4 widen_codes4(uint32_t c, float scale) {
  uint4 r;
  if constexpr (DT == HYB_BF16) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 3));
  }
  return r;
}

// Eight columns c0.. of a row of 16-bit elements; columns from k on are zero.
__device__ __forceinline__ uint4 load8_16(const uint16_t* row, int32_t c0, int32_t k) {
  if (c0 + 8 <= k) {
    const Bytes16 u = *reinterpret_cast<const Bytes16*>(row + c0);
    return make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i < k) w[i >> 1] |= uint32_t(row[c0 + i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// with_act for a gated product; f runs once with any activation for others.
template <bool GATED, typename F>
__device__ __forceinline__ void with_gated(int act, F f) {
  if constexpr (GATED)
    with_act(act, f);
  else
    f(std::integral_constant<int, HYB_ACT_SILU>());
}

// Sets of registers that a wavefront's codes of 512 columns take turns in: the
// next are loaded whole ahead of the products (two), or, with two weights, step by
// step into the registers that the products have done with (one: the gated kernels
// would need 145 registers, and 17408x5120 at 32 tokens takes 36.8 us instead of
// 31.9; a single weight's with one 8192x28672 at 64 tokens 67.9 instead of 60.2).
template <int P>
constexpr int kRing = P == 1 ? 2 : 1;

// Few tokens: one workgroup per panel (of each weight, gated), its wavefronts
// cut k.  A lane loads 16 bytes of codes a step (32 codes of its row, eight for
// each of four matrix instructions), 16 bytes of scales per four steps, and the
// wavefront MT tokens' 512 columns, which it keeps in LDS.  Bound by memory, and
// below ten microseconds by the depth of a launch: 14336x4096, one token 7.0 us for
// 31 MB (4.5 TB/s).
template <int DT, int MT, bool GATED, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q4_rows(Q4Args a) {
  constexpr int P = GATED ? 2 : 1;
  constexpr int kRow = 1024 + 16;  // a token's 512 columns, rows 4 banks apart
  constexpr int kOwn = MT * kRow > P * MT * 64 ? MT * kRow : P * MT * 64;
  __shared__ __attribute__((aligned(16))) char smem[WAVES * kOwn];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* xs = smem + wave * kOwn;
  const int64_t panel = blockIdx.x, tok0 = int64_t(blockIdx.y) * MT;
  const int32_t quads = (a.steps + 3) / 4;
  const int32_t q0 = quads * wave / WAVES, q1 = quads * (wave + 1) / WAVES;
  const int64_t row = panel * 16 + (lane & 15);

  __amdgpu_buffer_rsrc_t code_rsrc[P];
  const char* scale_at[P];
  int lift[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    code_rsrc[p] = make_rsrc(a.w[p].codes + panel * a.steps * kQ4StepBytes, a.steps * int32_t(kQ4StepBytes));
    scale_at[p] = a.w[p].scales + row * 16;
    lift[p] = DT == HYB_F16 ? kTopLift - int(a.w[p].tops[row]) : 0;
  }
  uint4 code[kRing<P>][P][4], scale[2][P], xr[MT];
  f32x4_t acc[P];
#pragma unroll
  for (int p = 0; p < P; ++p) acc[p] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto load_x = [&](int32_t q) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
      xr[t] = tok0 + t < a.m ? load8_16(a.x + (tok0 + t) * a.ldx, q * 512 + lane * 8, a.k) : make_uint4(0, 0, 0, 0);
  };
  auto load_scale = [&](int32_t q, uint4 (&sc)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) sc[p] = *reinterpret_cast<const uint4*>(scale_at[p] + int64_t(q) * a.rows16 * 16);
  };
  auto load_step = [&](int32_t step, uint4 (&c)[P][4], int s) {
#pragma unroll
    for (int p = 0; p < P; ++p)  // (steps behind the last lie behind the resource: zeros)
      c[p][s] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(code_rsrc[p], step * 1024 + lane * 16, 0, HYB_W_AUX));
  };
  const int t16 = lane & 15;
  const char* xb = xs + (t16 < MT ? t16 : MT - 1) * kRow + (lane >> 4) * 16;
  if (q0 < q1) {
    load_x(q0);
    load_scale(q0, scale[0]);
#pragma unroll
    for (int s = 0; s < 4; ++s) load_step(q0 * 4 + s, code[0], s);
  }
  auto quad = [&](int32_t q, auto turn) {
    constexpr int T = decltype(turn)::value, B = kRing<P> == 2 ? T : 0;
    const bool more = q + 1 < q1;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<uint4*>(xs + t * kRow + lane * 16) = xr[t];
    __builtin_amdgcn_wave_barrier();
    if (more) {
      load_x(q + 1);
      load_scale(q + 1, scale[1 - T]);
      if constexpr (kRing<P> == 2) {
#pragma unroll
        for (int s = 0; s < 4; ++s) load_step(q * 4 + 4 + s, code[1 - B], s);
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint4 b[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) b[h] = *reinterpret_cast<const uint4*>(xb + s * 256 + h * 64);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint4 cw = code[B][p][s];
        const uint32_t c[4] = {cw.x, cw.y, cw.z, cw.w};
        const uint32_t sw = s == 0 ? scale[T][p].x : s == 1 ? scale[T][p].y : s == 2 ? scale[T][p].z : scale[T][p].w;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          acc[p] = mfma16x16x32<DT>(widen_codes4<DT>(c[h], group_scale<DT>(sw, h, lift[p])), b[h], acc[p]);
      }
      if (kRing<P> == 1 && more) load_step(q * 4 + 4 + s, code[0], s);
    }
  };
  for (int32_t q = q0; q < q1; q += 2) {
    quad(q, std::integral_constant<int, 0>());
    if (q + 1 < q1) quad(q + 1, std::integral_constant<int, 1>());
  }
  // sums of the wavefronts, in order: [wave][weight][token][row]
  __builtin_amdgcn_wave_barrier();
  float* red = reinterpret_cast<float*>(xs);
  if (t16 < MT) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<f32x4_t*>(red + (p * MT + t16) * 16 + (lane >> 4) * 4) = acc[p];
  }
  __syncthreads();
  with_gated<GATED>(a.act, [&](auto act) {
    for (int i = threadIdx.x; i < MT * 16; i += 64 * WAVES) {
      const int t = i >> 4, r = i & 15;
      if (tok0 + t >= a.m || panel * 16 + r >= a.n) continue;
      float v[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        v[p] = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v[p] += reinterpret_cast<const float*>(smem + w * kOwn)[(p * MT + t) * 16 + r];
        if constexpr (DT == HYB_F16) v[p] = __builtin_ldexpf(v[p], int(a.w[p].tops[panel * 16 + r]) - kTopLift);
      }
      const float out = GATED ? act_value<decltype(act)::value>(v[0]) * v[P - 1] : v[0];
      store_out(a.y, a.ydt, (tok0 + t) * a.ldy + panel * 16 + r, out);
    }
  });
}

// Activations as panels (hyb_panel.h), rows behind m and columns behind k zero
// (read where they lie, 64 bytes of a row at a time, they cost a tile a fifth of its
// time): a wavefront per panel and four steps, whose eight loads are under way at once.
__global__ __launch_bounds__(256) void k_q4_pack_x(const uint16_t* __restrict__ x, int64_t ldx, int64_t m, int32_t k,
                                                   int32_t steps64, char* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t panel = blockIdx.x;
  const int32_t s = (int32_t(blockIdx.y) * 4 + wave) * 4;
  if (s >= steps64) return;
  const int64_t row = panel * 16 + (lane & 15);
  const int32_t c0 = s * 64 + (lane >> 4) * 8;
  uint4 u[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) u[h] = row < m ? load8_16(x + row * ldx, c0 + h * 32, k) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int h = 0; h < 8; ++h)
    if (s + h / 2 < steps64)
      *reinterpret_cast<uint4*>(out + (panel * steps64 + s) * 2048 + h * 1024 + lane * 16) = u[h];
}

// Four outputs j0.. of token `tok`: sums v (and u of the second weight).
__device__ __forceinline__ void q4_store4(const Q4Args& a, int64_t tok, int64_t j0, f32x4_t v) {
  if (tok >= a.m || j0 >= a.n) return;
  const int64_t at = tok * a.ldy + j0;
  if (j0 + 4 <= a.n) {
    if (a.ydt == HYB_F32) {
      const u32x4_t u = __builtin_bit_cast(u32x4_t, v);
      *reinterpret_cast<Bytes16*>(static_cast<float*>(a.y) + at) = Bytes16{{u[0], u[1], u[2], u[3]}};
    } else {
      const uint2 h = a.ydt == HYB_BF16 ? round16x4<HYB_BF16>(v[0], v[1], v[2], v[3])
                                        : round16x4<HYB_F16>(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<Bytes8*>(static_cast<uint16_t*>(a.y) + at) = Bytes8{{h.x, h.y}};
    }
    return;
  }
  for (int e = 0; e < 4; ++e)
    if (j0 + e < a.n) store_out(a.y, a.ydt, at + e, v[e]);
}

// Sums of rows j0.. of weight p in their own scale.
template <int DT>
__device__ __forceinline__ f32x4_t q4_lift(const Q4Args& a, int p, int64_t j0, f32x4_t v) {
  if constexpr (DT == HYB_F16) {
    // (rows behind the last have no outputs: any exponent)
    const uint32_t t = *reinterpret_cast<const uint32_t*>(a.w[p].tops + (j0 < a.rows16 ? j0 : a.rows16 - 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e], int((t >> (8 * e)) & 0xFFu) - kTopLift);
  }
  return v;
}

template <int DT, bool GATED, int ACT>
__device__ __forceinline__ f32x4_t q4_finish(const Q4Args& a, int64_t j0, f32x4_t v, f32x4_t u) {
  v = q4_lift<DT>(a, 0, j0, v);
  if constexpr (GATED) {
    u = q4_lift<DT>(a, 1, j0, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = act_value<ACT>(v[e]) * u[e];
  }
  return v;
}

// Up to a few hundred tokens on short matrices: eight panels (of each weight) per
// workgroup, one per wavefront, whose codes go from memory to its registers; 16
// BP tokens' activations, 512 columns at a time, come through LDS for all eight
// (from registers, in which a row at any alignment and the end of k cost nothing
// more).  The k of a workgroup's panels may be cut into parts, a workgroup each.
// Bound by memory with one block of tokens: 8192x28672, 13 tokens, eight parts 23.6-24.8
// us for 125 MB (5.0-5.3 TB/s), and 4.1 for the sums; gated 17408x5120, 16 tokens 21.0-22.4
// and 4.0.  With 64 tokens by the LDS, where each panel reads them all: 58 and 5, gated 43
// and 5 (every wavefront with its own activations, as in k_q4_rows, 413 and 194).
template <int DT, bool GATED, int BP>
__global__ __launch_bounds__(512) void k_q4_shared(Q4Args a) {
  constexpr int P = GATED ? 2 : 1;
  constexpr int kX = BP * 16384;       // 512 columns
  constexpr int kLoads = BP * 16 / 8;  // 1 KiB of them per wavefront
  extern __shared__ __attribute__((aligned(1024))) char q4_smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t part = int32_t(blockIdx.y);
  const int32_t quads = (a.steps + 3) / 4;
  const int32_t q0 = int32_t(int64_t(quads) * part / a.parts), q1 = int32_t(int64_t(quads) * (part + 1) / a.parts);
  const int64_t panels = a.rows16 / 16, mine = int64_t(blockIdx.x) * 8 + wave;
  const int64_t tok0 = int64_t(blockIdx.z) * (BP * 16);
  // (a wavefront behind the last panel multiplies the last one again)
  const int64_t panel = mine < panels ? mine : panels - 1;
  const int64_t row = panel * 16 + (lane & 15);

  __amdgpu_buffer_rsrc_t code_rsrc[P];
  const char* scale_at[P];
  int lift[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    code_rsrc[p] = make_rsrc(a.w[p].codes + panel * a.steps * kQ4StepBytes, a.steps * int32_t(kQ4StepBytes));
    scale_at[p] = a.w[p].scales + row * 16;
    lift[p] = DT == HYB_F16 ? kTopLift - int(a.w[p].tops[row]) : 0;
  }
  // x: KiB c of a quad is half c % 2 of 64-column step c / 2 % 8 of token panel
  // c / 16; this wavefront's are wave * kLoads ..
  uint4 xr[kLoads];
  auto load_x = [&](int32_t q) {
#pragma unroll
    for (int t = 0; t < kLoads; ++t) {
      const int c = wave * kLoads + t;
      // (a lane behind the last token or at the row's end loads the last token's or
      // the row's last eight columns, so that no load branches)
      const int64_t tok = tok0 + (c >> 4) * 16 + (lane & 15);
      const int32_t col = q * 512 + (c & 15) * 32 + (lane >> 4) * 8;
      const Bytes16 u = *reinterpret_cast<const Bytes16*>(a.x + (tok < a.m ? tok : a.m - 1) * a.ldx +
                                                          (col < a.k - 8 ? col : a.k - 8));
      xr[t] = make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
    }
  };
  auto store_x = [&](int32_t q) {
    if ((q + 1) * 512 > a.k) {
#pragma unroll
      for (int t = 0; t < kLoads; ++t)
        xr[t] = move_down(xr[t], q * 512 + ((wave * kLoads + t) & 15) * 32 + (lane >> 4) * 8 - (a.k - 8));
    }
#pragma unroll
    for (int t = 0; t < kLoads; ++t)
      *reinterpret_cast<uint4*>(q4_smem + (q & 1) * kX + (wave * kLoads + t) * 1024 + lane * 16) = xr[t];
  };
  uint4 code[kRing<P>][P][4], scale[2][P];
  auto load_scale = [&](int32_t q, uint4 (&sc)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) sc[p] = *reinterpret_cast<const uint4*>(scale_at[p] + int64_t(q) * a.rows16 * 16);
  };
  auto load_step = [&](int32_t step, uint4 (&c)[P][4], int s) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      c[p][s] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(code_rsrc[p], step * 1024 + lane * 16, 0, HYB_W_AUX));
  };
  f32x4_t acc[P][BP];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < BP; ++j) acc[p][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (q0 < q1) {
    load_x(q0);
    load_scale(q0, scale[0]);
#pragma unroll
    for (int s = 0; s < 4; ++s) load_step(q0 * 4 + s, code[0], s);
  }
  auto quad = [&](int32_t q, auto turn) {
    constexpr int T = decltype(turn)::value, B = kRing<P> == 2 ? T : 0;
    const bool more = q + 1 < q1;
    // (this half of the LDS was read ahead of the last barrier)
    store_x(q);
    if (more) {
      load_x(q + 1);
      load_scale(q + 1, scale[1 - T]);
      if constexpr (kRing<P> == 2) {
#pragma unroll
        for (int s = 0; s < 4; ++s) load_step(q * 4 + 4 + s, code[1 - B], s);
      }
    }
    __syncthreads();
    const char* xs = q4_smem + (q & 1) * kX + lane * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint4 b[BP];
#pragma unroll
        for (int j = 0; j < BP; ++j) b[j] = *reinterpret_cast<const uint4*>(xs + j * 16384 + s * 4096 + h * 1024);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint4 cw = code[B][p][s];
          const uint32_t c = h == 0 ? cw.x : h == 1 ? cw.y : h == 2 ? cw.z : cw.w;
          const uint32_t sw = s == 0 ? scale[T][p].x : s == 1 ? scale[T][p].y : s == 2 ? scale[T][p].z : scale[T][p].w;
          const uint4 w = widen_codes4<DT>(c, group_scale<DT>(sw, h, lift[p]));
#pragma unroll
          for (int j = 0; j < BP; ++j) acc[p][j] = mfma16x16x32<DT>(w, b[j], acc[p][j]);
        }
      }
      if (kRing<P> == 1 && more) load_step(q * 4 + 4 + s, code[0], s);
    }
  };
  for (int32_t q = q0; q < q1; q += 2) {
    quad(q, std::integral_constant<int, 0>());
    if (q + 1 < q1) quad(q + 1, std::integral_constant<int, 1>());
  }
  const int64_t block = int64_t(blockIdx.z) * gridDim.x + blockIdx.x;
  if (a.parts > 1) {
    f32x4_t* out = a.ws + ((block * a.parts + part) * 8 + wave) * (P * BP * 64) + lane;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < BP; ++j) out[(p * BP + j) * 64] = acc[p][j];
    return;
  }
  if (mine >= panels) return;
  const int64_t j0 = panel * 16 + (lane >> 4) * 4;
  with_gated<GATED>(a.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < BP; ++j)
      q4_store4(a, tok0 + j * 16 + (lane & 15), j0,
                q4_finish<DT, GATED, decltype(act)::value>(a, j0, acc[0][j], acc[P - 1][j]));
  });
}

// Adds the parts of k_q4_shared in order: one thread per four outputs.
template <int DT, bool GATED, int BP>
__global__ __launch_bounds__(256) void k_q4_shared_sum(Q4Args a) {
  constexpr int P = GATED ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const int c = int(blockIdx.y) * 4 + (threadIdx.x >> 6), wave = c / BP, j = c % BP;
  const int64_t j0 = (int64_t(blockIdx.x) * 8 + wave) * 16 + (lane >> 4) * 4;
  const int64_t block = int64_t(blockIdx.z) * gridDim.x + blockIdx.x, tok = (int64_t(blockIdx.z) * BP + j) * 16 + (lane & 15);
  if (tok >= a.m || j0 >= a.n) return;
  f32x4_t v[2];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const f32x4_t* at = a.ws + (block * a.parts * 8 + wave) * (P * BP * 64) + (p * BP + j) * 64 + lane;
    f32x4_t sum = at[0];
#pragma unroll 4
    for (int t = 1; t < a.parts; ++t) {
      const f32x4_t o = at[int64_t(t) * 8 * (P * BP * 64)];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += o[e];
    }
    v[p] = sum;
  }
  with_gated<GATED>(a.act, [&](auto act) {
    q4_store4(a, tok, j0, q4_finish<DT, GATED, decltype(act)::value>(a, j0, v[0], v[P - 1]));
  });
}

// More tokens: AP panels of codes x BP panels of tokens through LDS, WA x WB
// wavefronts.  Codes stay 4-bit up to the registers, where two instructions'
// worth of eight are widened, scale included, for every BP / WB x 2 matrix
// instructions they feed.  A step is 64 columns of x; codes come 128 columns at
// a time (half the panels in each of two steps), scales 512.  Bound by the matrix
// units and LDS: 17408x5120, 2048 tokens 273-292 us in a kernel trace, 1.25-1.34 Pflop/s
// (the whole call takes 262-284 in a loop; a dense bf16 product of 8192 cubed reaches
// 1.51), gated 556 (522 the call), fp16 697 (612).
template <int DT, bool GATED, int AP, int BP, int WA, int WB>
struct Q4Tile {
  static constexpr int kWaves = WA * WB;
  static constexpr int kA = AP / WA, kB = BP / WB;
  static constexpr int kCodes = AP * 1024, kScales = AP * 256, kX = BP * 2048;
  static constexpr int kStages = 2 * (kCodes + kScales + kX);
  static constexpr int kOutA = GATED ? kA / 2 : kA;
  static constexpr int kOutBytes = kWaves * kOutA * kB * 512;
  static constexpr int kLds = kStages > kOutBytes ? kStages : kOutBytes;
  static constexpr int kPanels = GATED ? AP / 2 : AP;  // of each weight
  static constexpr int kLoadsX = BP * 2 / kWaves;
  static_assert(AP / 2 == kWaves && BP * 2 % kWaves == 0 && AP % WA == 0 && BP % WB == 0, "even split");

  __device__ static void run(const Q4Args& a, int32_t ab, int32_t bb, int32_t s0, int32_t s1, char* smem,
                             f32x4_t (&acc)[kA][kB]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wa = wave % WA, wb = wave / WA;
    const uint32_t base = __builtin_amdgcn_readfirstlane(panel_lds_addr(smem));
    constexpr int kAtScales = 2 * kCodes, kAtX = kAtScales + 2 * kScales;
    const int64_t panels = a.rows16 / 16, first = int64_t(ab) * kPanels;
    const int64_t exist = panels - first < kPanels ? panels - first : kPanels;

    // codes: chunk c is panel c of the tile (gated: the second weight's from
    // AP / 2 on); this wavefront's are `wave` and `wave + AP / 2`
    const int c0 = wave, c1 = wave + AP / 2;
    auto code_rsrc = [&](int c) {
      const char* from = GATED && c >= AP / 2 ? a.w[1].codes : a.w[0].codes;
      return panel_srd(from + first * a.steps * kQ4StepBytes, uint32_t(exist * a.steps * kQ4StepBytes));
    };
    const srd4_t cr0 = code_rsrc(c0), cr1 = code_rsrc(c1);
    const int32_t pitch = a.steps * int32_t(kQ4StepBytes);
    const int32_t co0 = c0 * pitch + lane * 16, co1 = (GATED ? c1 - AP / 2 : c1) * pitch + lane * 16;
    auto issue_codes = [&](int32_t d, int half) {
      const uint32_t dst = base + (d & 1) * kCodes;
      if (half == 0)
        panel_dma16(cr0, __builtin_amdgcn_readfirstlane(dst + c0 * 1024), co0 + d * 1024);
      else
        panel_dma16(cr1, __builtin_amdgcn_readfirstlane(dst + c1 * 1024), co1 + d * 1024);
    };
    // scales: 1 KiB is four panels
    auto issue_scales = [&](int32_t q) {
      if (wave >= AP / 4) return;
      const int c = wave;
      const bool second = GATED && c >= AP / 8;
      const char* from = second ? a.w[1].scales : a.w[0].scales;
      const srd4_t r = panel_srd(from + (int64_t(q) * a.rows16 + first * 16) * 16, uint32_t(exist * 256));
      panel_dma16(r, __builtin_amdgcn_readfirstlane(base + kAtScales + (q & 1) * kScales + c * 1024), (second ? c - AP / 8 : c) * 1024 + lane * 16);
    };
    // x: chunk c is half c % 2 of panel c / 2
    const int64_t tok0 = int64_t(bb) * BP * 16, left = a.m - tok0;
    const int64_t rows = left < BP * 16 ? left : BP * 16;
    const srd4_t xr = panel_srd(a.xt + int64_t(bb) * BP * a.x_panel, uint32_t((rows + 15) / 16 * a.x_panel));
    auto issue_x = [&](int32_t s) {
      const uint32_t dst = base + kAtX + (s & 1) * kX;
#pragma unroll
      for (int t = 0; t < kLoadsX; ++t) {
        const int c = wave * kLoadsX + t;
        panel_dma16(xr, __builtin_amdgcn_readfirstlane(dst + c * 1024),
                    int32_t((c >> 1) * a.x_panel) + s * 2048 + (c & 1) * 1024 + lane * 16);
      }
    };
    // panel i of this wavefront in the tile's order
    auto panel_of = [&](int i) {
      if constexpr (GATED) return i < kA / 2 ? wa * (kA / 2) + i : AP / 2 + wa * (kA / 2) + i - kA / 2;
      return wa * kA + i;
    };
    int lift[kA];
#pragma unroll
    for (int i = 0; i < kA; ++i) {
      lift[i] = 0;
      if constexpr (DT == HYB_F16) {
        const int p = panel_of(i);
        const bool second = GATED && p >= AP / 2;
        const int64_t row = (first + (second ? p - AP / 2 : p)) * 16 + (lane & 15);
        if (row < a.rows16) lift[i] = kTopLift - int(a.w[second ? 1 : 0].tops[row]);
      }
#pragma unroll
      for (int j = 0; j < kB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    if (s0 >= s1) return;
    issue_x(s0);
    issue_codes(s0 >> 1, 0);
    issue_codes(s0 >> 1, 1);
    issue_scales(s0 >> 3);

    uint32_t sw[kA];
#pragma unroll
    for (int i = 0; i < kA; ++i) sw[i] = 0;
    auto compute = [&](int32_t s, auto phase) {
      constexpr int kPhase = decltype(phase)::value;  // s % 4
      constexpr int half = kPhase & 1;
      const char* codes = smem + ((kPhase >> 1) & 1) * kCodes + lane * 16 + half * 8;
      const char* xs = smem + kAtX + half * kX + lane * 16;
      if constexpr (half == 0) {
        const char* sc = smem + kAtScales + ((s >> 3) & 1) * kScales + (lane & 15) * 16 + ((s >> 1) & 3) * 4;
#pragma unroll
        for (int i = 0; i < kA; ++i) sw[i] = *reinterpret_cast<const uint32_t*>(sc + panel_of(i) * 256);
      }
      uint2 c = *reinterpret_cast<const uint2*>(codes + panel_of(0) * 1024);
      uint4 b[kB][2];
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        b[j][0] = *reinterpret_cast<const uint4*>(xs + (wb * kB + j) * 2048);
        b[j][1] = *reinterpret_cast<const uint4*>(xs + (wb * kB + j) * 2048 + 1024);
      }
      if (s + 1 < s1) issue_x(s + 1);
      const int32_t d = (s >> 1) + 1;
      if (2 * d < s1) issue_codes(d, half);
      if (kPhase == 0 && (s & 7) == 0 && s + 8 < s1) issue_scales((s >> 3) + 1);
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        const uint2 was = c;
        if (i + 1 < kA) c = *reinterpret_cast<const uint2*>(codes + panel_of(i + 1) * 1024);
        const uint4 a0 = widen_codes4<DT>(was.x, group_scale<DT>(sw[i], 2 * half, lift[i]));
        const uint4 a1 = widen_codes4<DT>(was.y, group_scale<DT>(sw[i], 2 * half + 1, lift[i]));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kB; ++j) acc[i][j] = mfma16x16x32<DT>(a0, b[j][0], acc[i][j]);
#pragma unroll
        for (int j = 0; j < kB; ++j) acc[i][j] = mfma16x16x32<DT>(a1, b[j][1], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int32_t q = s0; q < s1; q += 4) {
      auto one = [&](auto phase) {
        const int32_t s = q + decltype(phase)::value;
        if (s >= s1) return;
        panel_wait<0>();
        __syncthreads();
        compute(s, phase);
      };
      one(std::integral_constant<int, 0>());
      one(std::integral_constant<int, 1>());
      one(std::integral_constant<int, 2>());
      one(std::integral_constant<int, 3>());
    }
  }
};

// Column steps of a part: whole multiples of eight (the scales' 512 columns).
__device__ __forceinline__ int32_t q4_part_step(int32_t steps64, int32_t part, int32_t parts) {
  const int32_t octs = (steps64 + 7) / 8;
  const int32_t s = int32_t(int64_t(octs) * part / parts) * 8;
  return s < steps64 ? s : steps64;
}

template <int DT, bool GATED, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void k_q4_tile(Q4Args a) {
  typedef Q4Tile<DT, GATED, AP, BP, WA, WB> T;
  extern __shared__ __attribute__((aligned(1024))) char q4_smem[];
  const int32_t na = int32_t((a.rows16 / 16 + T::kPanels - 1) / T::kPanels);
  const int32_t nb = int32_t((a.m + BP * 16 - 1) / (BP * 16));
  const int32_t id = int32_t(blockIdx.x), rest = id - a.whole;
  const bool cut = rest >= 0;
  const int32_t part = cut ? rest % a.parts : 0;
  int32_t ab, bb;
  panel_block(cut ? a.whole + rest / a.parts : panel_order(id, a.whole), na, nb, ab, bb);
  f32x4_t acc[T::kA][T::kB];
  T::run(a, ab, bb, cut ? q4_part_step(a.steps64, part, a.parts) : 0,
         cut ? q4_part_step(a.steps64, part + 1, a.parts) : a.steps64, q4_smem, acc);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  if (cut) {
    f32x4_t* out = a.ws + (int64_t(rest) * T::kWaves + wave) * (T::kA * T::kB * 64) + lane;
#pragma unroll
    for (int i = 0; i < T::kA; ++i)
#pragma unroll
      for (int j = 0; j < T::kB; ++j) out[(i * T::kB + j) * 64] = acc[i][j];
    return;
  }
  const int64_t col0 = (int64_t(ab) * T::kPanels + wa * T::kOutA) * 16;
  const int64_t row0 = (int64_t(bb) * BP + wb * T::kB) * 16;
  // A gated tile's outputs take the place of its first sums, so that what follows is
  // there once and not for each activation.  (With three copies of it the loops over
  // the sums were too long to unroll, and the sums lay in memory throughout: gated
  // 17408x5120, 2048 tokens 6955 us.)
  if constexpr (GATED)
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < T::kOutA; ++i) {
#pragma unroll
        for (int j = 0; j < T::kB; ++j)
          acc[i][j] = q4_finish<DT, GATED, decltype(act)::value>(a, col0 + i * 16 + (lane >> 4) * 4, acc[i][j],
                                                                 acc[i + T::kA / 2][j]);
        __builtin_amdgcn_sched_barrier(0);  // (fp16: the rows' exponents of one i at a time)
      }
    });
  auto value = [&](int i, int j) {
    if constexpr (GATED) return acc[i][j];
    return q4_lift<DT>(a, 0, col0 + i * 16 + (lane >> 4) * 4, acc[i][j]);
  };
  if (a.ydt == HYB_F32) {
#pragma unroll
    for (int j = 0; j < T::kB; ++j)
#pragma unroll
      for (int i = 0; i < T::kOutA; ++i)
        q4_store4(a, row0 + j * 16 + (lane & 15), col0 + i * 16 + (lane >> 4) * 4, value(i, j));
    return;
  }
  __syncthreads();  // the tile's LDS stages are free
  const bool bf = a.ydt == HYB_BF16;
  panel_rows16<T::kOutA, T::kB>(
      q4_smem + wave * (T::kOutA * T::kB * 512), lane, lane & 15,
      [&](int i, int j) {
        const f32x4_t v = value(i, j);
        return bf ? round16x4<HYB_BF16>(v[0], v[1], v[2], v[3]) : round16x4<HYB_F16>(v[0], v[1], v[2], v[3]);
      },
      [&](int r, int c, uint4 u) {
        const int64_t tok = row0 + r, col = col0 + c;
        if (tok >= a.m || col >= a.n) return;
        uint16_t* p = static_cast<uint16_t*>(a.y) + tok * a.ldy + col;
        if (col + 8 <= a.n) {
          *reinterpret_cast<Bytes16*>(p) = Bytes16{{u.x, u.y, u.z, u.w}};
        } else {
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          for (int e = 0; e < 8; ++e)
            if (col + e < a.n) p[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
        }
      });
}

// Adds the parts of a tile in order and stores the outputs: one thread per four
// outputs, in the order of the tile's registers.
template <int DT, bool GATED, int AP, int BP, int WA, int WB>
__global__ __launch_bounds__(256) void k_q4_sum(Q4Args a) {
  typedef Q4Tile<DT, GATED, AP, BP, WA, WB> T;
  constexpr int kEach = T::kWaves * T::kOutA * T::kB;  // of 64 lanes, a tile
  const int32_t na = int32_t((a.rows16 / 16 + T::kPanels - 1) / T::kPanels);
  const int32_t nb = int32_t((a.m + BP * 16 - 1) / (BP * 16));
  int32_t ab, bb;
  panel_block(a.whole + int32_t(blockIdx.x), na, nb, ab, bb);
  const int lane = threadIdx.x & 63;
  const int c = int(blockIdx.y) * 4 + (threadIdx.x >> 6);
  if (c >= kEach) return;
  const int wave = c / (T::kOutA * T::kB), i = c / T::kB % T::kOutA, j = c % T::kB;
  const int64_t j0 = (int64_t(ab) * T::kPanels + wave % WA * T::kOutA + i) * 16 + (lane >> 4) * 4;
  const int64_t tok = (int64_t(bb) * BP + wave / WA * T::kB + j) * 16 + (lane & 15);
  if (tok >= a.m || j0 >= a.n) return;
  f32x4_t v[2];
#pragma unroll
  for (int p = 0; p < (GATED ? 2 : 1); ++p) {
    const f32x4_t* at = a.ws + (int64_t(blockIdx.x) * a.parts * T::kWaves + wave) * (T::kA * T::kB * 64) +
                        ((i + p * (T::kA / 2)) * T::kB + j) * 64 + lane;
    f32x4_t sum = at[0];
#pragma unroll 4
    for (int t = 1; t < a.parts; ++t) {
      const f32x4_t o = at[int64_t(t) * T::kWaves * (T::kA * T::kB * 64)];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += o[e];
    }
    v[p] = sum;
  }
  with_gated<GATED>(a.act, [&](auto act) {
    q4_store4(a, tok, j0, q4_finish<DT, GATED, decltype(act)::value>(a, j0, v[0], v[GATED ? 1 : 0]));
  });
}

// Zeros (k = 0).
__global__ __launch_bounds__(256) void k_q4_zero(Q4Args a) {
  const int64_t j = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (j >= a.n) return;
  for (int64_t t = blockIdx.y; t < a.m; t += gridDim.y) store_out(a.y, a.ydt, t * a.ldy + j, 0.f);
}

// ----------------------------------------------------------------- launches --

template <int DT, int MT, bool GATED>
hipError_t run_rows(const Q4Args& a, hipStream_t s) {
  const dim3 grid(unsigned(a.rows16 / 16), unsigned((a.m + MT - 1) / MT));
  if (a.steps > 16)
    hipLaunchKernelGGL((k_q4_rows<DT, MT, GATED, 8>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((k_q4_rows<DT, MT, GATED, 4>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DT, bool GATED, int AP, int BP, int WA, int WB>
hipError_t run_tile(const Q4Args& a, hipStream_t s) {
  typedef Q4Tile<DT, GATED, AP, BP, WA, WB> T;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_q4_tile<DT, GATED, AP, BP, WA, WB>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
  if (e != hipSuccess) return e;
  const int64_t na = (a.rows16 / 16 + T::kPanels - 1) / T::kPanels, nb = (a.m + BP * 16 - 1) / (BP * 16);
  const int64_t rest = na * nb - a.whole;
  hipLaunchKernelGGL((k_q4_tile<DT, GATED, AP, BP, WA, WB>), dim3(unsigned(a.whole + rest * a.parts)),
                     dim3(64 * T::kWaves), T::kLds, s, a);
  if ((e = hipGetLastError()) != hipSuccess || rest == 0) return e;
  constexpr int kEach = T::kWaves * T::kOutA * T::kB;
  hipLaunchKernelGGL((k_q4_sum<DT, GATED, AP, BP, WA, WB>), dim3(unsigned(rest), unsigned((kEach + 3) / 4)), dim3(256), 0, s,
                     a);
  return hipGetLastError();
}

template <int DT, bool GATED, int BP>
hipError_t run_shared(const Q4Args& a, hipStream_t s) {
  constexpr int kLds = 2 * BP * 16384;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_q4_shared<DT, GATED, BP>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  const unsigned blocks = unsigned((a.rows16 / 16 + 7) / 8), tokens = unsigned((a.m + BP * 16 - 1) / (BP * 16));
  hipLaunchKernelGGL((k_q4_shared<DT, GATED, BP>), dim3(blocks, unsigned(a.parts), tokens), dim3(512), kLds, s, a);
  if ((e = hipGetLastError()) != hipSuccess || a.parts <= 1) return e;
  hipLaunchKernelGGL((k_q4_shared_sum<DT, GATED, BP>), dim3(blocks, 2 * BP, tokens), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DT, bool GATED>
hipError_t run_product(Q4Args& a, const Q4Route& r, char* ws, hipStream_t s) {
  if (r.ap == 0) {
    if (a.m == 1) return run_rows<DT, 1, GATED>(a, s);
    if (a.m == 2) return run_rows<DT, 2, GATED>(a, s);
    return run_rows<DT, 4, GATED>(a, s);
  }
  a.ws = reinterpret_cast<f32x4_t*>(ws + q4_pack_bytes(r, a.k, a.m));
  a.parts = r.parts;
  a.whole = int32_t(r.whole);
  if (r.bp == 1) return run_shared<DT, GATED, 1>(a, s);
  if (r.bp == 2) return run_shared<DT, GATED, 2>(a, s);
  if (r.bp == 4) return run_shared<DT, GATED, 4>(a, s);
  hipLaunchKernelGGL(k_q4_pack_x, dim3(unsigned((a.m + 15) / 16), unsigned((a.steps64 + 15) / 16)), dim3(256), 0, s, a.x,
                     a.ldx, a.m, a.k, a.steps64, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.xt = ws;
  a.x_panel = int64_t(a.steps64) * 2048;
  if (r.bp == 8) return run_tile<DT, GATED, 16, 8, 4, 2>(a, s);
  return run_tile<DT, GATED, 16, 16, 2, 4>(a, s);
}

Q4Weight weight_of(const hyb_q4& w, int64_t n, int64_t k) {
  const char* scales = static_cast<const char*>(w.scales);
  return Q4Weight{static_cast<const char*>(w.codes), scales,
                  reinterpret_cast<const uint8_t*>(scales) + q4_quads(k) * q4_rows16(n) * 16};
}

}  // namespace

hipError_t launch_q4_quantize(const void* a, int dtype, int64_t n, int64_t k, int64_t lda, const hyb_q4& dst,
                              hipStream_t s) {
  const int64_t rows16 = q4_rows16(n);
  const int32_t steps = int32_t(q4_steps(k));
  const dim3 grid(unsigned(rows16 / 16));
  char* codes = static_cast<char*>(dst.codes);
  char* scales = static_cast<char*>(dst.scales);
  if (dtype == HYB_F32)
    hipLaunchKernelGGL((k_q4_quantize<HYB_F32>), grid, dim3(256), 0, s, a, n, int32_t(k), lda, steps, rows16, codes, scales);
  else if (dtype == HYB_BF16)
    hipLaunchKernelGGL((k_q4_quantize<HYB_BF16>), grid, dim3(256), 0, s, a, n, int32_t(k), lda, steps, rows16, codes, scales);
  else
    hipLaunchKernelGGL((k_q4_quantize<HYB_F16>), grid, dim3(256), 0, s, a, n, int32_t(k), lda, steps, rows16, codes, scales);
  return hipGetLastError();
}

hipError_t launch_q4_dequantize(const hyb_q4& src, int64_t n, int64_t k, void* a, int dtype, int64_t lda,
                                hipStream_t s) {
  const int64_t rows16 = q4_rows16(n);
  const int32_t steps = int32_t(q4_steps(k));
  const dim3 grid(unsigned(rows16 / 16), unsigned((steps + 3) / 4));
  const char* codes = static_cast<const char*>(src.codes);
  const char* scales = static_cast<const char*>(src.scales);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, codes, scales, n, int32_t(k), lda, steps, rows16, a);
  };
  // 16-bit rows that begin within 64 bytes leave parts of lines at both ends, which the
  // caches join: 28672x8192, row stride 8193 164 us (around them 196), 8200 168 (178);
  // 8224 182 (143), 8192 144 (95)
  const bool stream = n * k * 2 > kStreamBytes && (reinterpret_cast<uintptr_t>(a) | uintptr_t(lda * 2)) % 64 == 0;
  if (dtype == HYB_F32)
    go(&k_q4_dequantize<HYB_F32, false>);
  else if (dtype == HYB_BF16)
    stream ? go(&k_q4_dequantize<HYB_BF16, true>) : go(&k_q4_dequantize<HYB_BF16, false>);
  else
    stream ? go(&k_q4_dequantize<HYB_F16, true>) : go(&k_q4_dequantize<HYB_F16, false>);
  return hipGetLastError();
}

hipError_t launch_q4_product(const hyb_q4& w, const hyb_q4* up, int act, int64_t n, int64_t k, const void* x,
                             int x_dtype, int64_t m, int64_t ldx, void* y, int y_dtype, int64_t ldy, char* ws,
                             hipStream_t s) {
  Q4Args a{};
  a.rows16 = q4_rows16(n);
  a.steps = int32_t(q4_steps(k));
  a.steps64 = int32_t((k + 63) / 64);
  a.n = int32_t(n);
  a.k = int32_t(k);
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.m = m;
  a.y = y;
  a.ldy = ldy;
  a.ydt = y_dtype;
  a.act = act;
  if (k == 0) {
    hipLaunchKernelGGL(k_q4_zero, dim3(unsigned((n + 255) / 256), unsigned(m < 65535 ? m : 65535)), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  a.w[0] = weight_of(w, n, k);
  if (up) a.w[1] = weight_of(*up, n, k);
  const Q4Route r = q4_route(n, k, m, up ? 2 : 1, device_cus());
  if (x_dtype == HYB_BF16)
    return up ? run_product<HYB_BF16, true>(a, r, ws, s) : run_product<HYB_BF16, false>(a, r, ws, s);
  return up ? run_product<HYB_F16, true>(a, r, ws, s) : run_product<HYB_F16, false>(a, r, ws, s);
}

}  // namespace hyb
