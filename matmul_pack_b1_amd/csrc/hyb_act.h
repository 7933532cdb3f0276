// Activations of the gated projection and their derivatives, fp32.
//   silu       g s,       s = 1 / (1 + exp(-g))
//   gelu       g Phi(g),  Phi the normal distribution function
//   gelu_tanh  g (1 + tanh(y)) / 2 = g s,  y = c (g + 0.044715 g^3),
//              c = sqrt(2 / pi), s = 1 / (1 + exp(-2 y))
#ifndef HYB_ACT_H_
#define HYB_ACT_H_

#include <type_traits>

#include "hyb_device.h"
#include "../../include/hyb_gated.h"

namespace hyb {
namespace {

__device__ __forceinline__ float act_sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Phi from the complementary error function of |g|, which keeps the small
// values of the left tail (1 + erf loses them from g = -4 on): the rational
// Chebyshev fit of Numerical Recipes (Press et al., 6.2, "erfcc"),
// erfc(x) = t exp(-x^2 + P(t)), t = 1 / (1 + x / 2), off by at most 1.2e-7
// relative for every x >= 0.
__device__ __forceinline__ float act_phi(float g) {
  const float x = __builtin_fabsf(g) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.f));
  float p = 0.17087277f;
  p = __builtin_fmaf(p, t, -0.82215223f);
  p = __builtin_fmaf(p, t, 1.48851587f);
  p = __builtin_fmaf(p, t, -1.13520398f);
  p = __builtin_fmaf(p, t, 0.27886807f);
  p = __builtin_fmaf(p, t, -0.18628806f);
  p = __builtin_fmaf(p, t, 0.09678418f);
  p = __builtin_fmaf(p, t, 0.37409196f);
  p = __builtin_fmaf(p, t, 1.00002368f);
  p = __builtin_fmaf(p, t, -1.26551223f);
  const float c = 0.5f * t * __builtin_amdgcn_exp2f(__builtin_fmaf(-x, x, p) * 1.4426950408889634f);
  return g < 0.f ? c : 1.f - c;
}

constexpr float kGeluC = 0.79788456080286536f;

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == HYB_ACT_SILU) return g * act_sigmoid(g);
  if constexpr (ACT == HYB_ACT_GELU_TANH) return g * act_sigmoid(2.f * kGeluC * g * __builtin_fmaf(0.044715f * g, g, 1.f));
  return g * act_phi(g);
}

// The value in *a and the derivative.
template <int ACT>
__device__ __forceinline__ float act_slope(float g, float* a) {
  if constexpr (ACT == HYB_ACT_SILU) {
    const float s = act_sigmoid(g);
    *a = g * s;
    return __builtin_fmaf(*a, 1.f - s, s);
  } else if constexpr (ACT == HYB_ACT_GELU_TANH) {
    const float gg = 0.044715f * g * g;
    const float s = act_sigmoid(2.f * kGeluC * g * (gg + 1.f));
    *a = g * s;
    // (where s has reached 0 or 1 the polynomial may have overflowed)
    const float t = s * (1.f - s);
    return t == 0.f ? s : __builtin_fmaf(g * t, 2.f * kGeluC * __builtin_fmaf(3.f, gg, 1.f), s);
  } else {
    const float p = act_phi(g);
    *a = g * p;
    // exp(-g^2 / 2) / sqrt(2 pi)
    const float d = 0.3989422804014327f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
    return d == 0.f ? p : __builtin_fmaf(g, d, p);
  }
}

// f(integral constant of the activation): one branch a kernel.  (At every element
// of a tile the three bodies, unrolled 64 times, did not fit the instruction cache:
// gated 17408x5120, 2048 tokens, five rounds of tiles, 728 us instead of 689.)
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == HYB_ACT_SILU)
    f(std::integral_constant<int, HYB_ACT_SILU>());
  else if (act == HYB_ACT_GELU)
    f(std::integral_constant<int, HYB_ACT_GELU>());
  else
    f(std::integral_constant<int, HYB_ACT_GELU_TANH>());
}

}  // namespace
}  // namespace hyb

#endif  // HYB_ACT_H_
