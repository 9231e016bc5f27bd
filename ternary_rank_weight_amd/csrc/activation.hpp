// The gated block's activations and their slopes, in fp32.
//   silu      g / (1 + exp(-g))
//   gelu      g (1 + erf(g / sqrt 2)) / 2
//   gelu_tanh g (1 + tanh(z)) / 2 = g / (1 + exp(-2 z)),  z = sqrt(2 / pi) (g + 0.044715 g^3)
// Each holds over the whole fp32 range: exp of a large argument is inf, and
// the quotient by it 0.
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/externd.h"

namespace externd {

__device__ __forceinline__ float sigmoid_f32(float z) { return 1.f / (1.f + expf(-z)); }

// Twice the tanh form's z, and its slope in g.
__device__ __forceinline__ float gelu_2z(float g) { return 1.5957691216057308f * g * (1.f + 0.044715f * g * g); }
__device__ __forceinline__ float gelu_2z_slope(float g) { return 1.5957691216057308f * (1.f + 0.134145f * g * g); }

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == EXTERND_ACT_SILU) return g * sigmoid_f32(g);
  else if constexpr (ACT == EXTERND_ACT_GELU) return 0.5f * g * erfcf(-0.7071067811865476f * g);
  else return g * sigmoid_f32(gelu_2z(g));
}

__device__ __forceinline__ float act_value(int act, float g) {
  if (act == EXTERND_ACT_SILU) return act_value<EXTERND_ACT_SILU>(g);
  if (act == EXTERND_ACT_GELU) return act_value<EXTERND_ACT_GELU>(g);
  return act_value<EXTERND_ACT_GELU_TANH>(g);
}

// The same for results that are rounded to 16 bits: hardware reciprocal and
// exponential.  Their relative error is a few 2^-24, and 2^-23 of the exponent's size more, whose
// rounding the exponential passes on: 1e-6 at an exponent of 8, 1e-5 at 80.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
// (1 + erf(g / sqrt 2)) / 2.  The tail past x = |g| is exp(-x^2 / 2) times a function that falls
// slowly, a polynomial in 1 / (1 + 0.265 x) fitted to erfcx(x / sqrt 2) / 2 on 0 <= x <= 14.5
// (6.3e-7 relative; farther out the exponential is 0): the tail keeps its relative
// error, 2e-6 up to x = 5, where one minus erf would keep none.
__device__ __forceinline__ float normal_cdf_fast(float g) {
  const float x = fabsf(g);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.265f, x, 1.f));
  float r = -0.0677870363f;
  r = fmaf(r, t, 0.195273116f);
  r = fmaf(r, t, -0.0663629249f);
  r = fmaf(r, t, 0.142493337f);
  r = fmaf(r, t, 0.0829465911f);
  r = fmaf(r, t, 0.107836783f);
  r = fmaf(r, t, 0.105599836f);
  const float tail = r * t * __builtin_amdgcn_exp2f(-0.7213475204444817f * x * x);
  return g < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_fast(float g) {
  if constexpr (ACT == EXTERND_ACT_SILU) return g * sigmoid_fast(g);
  else if constexpr (ACT == EXTERND_ACT_GELU) return g * normal_cdf_fast(g);
  else return g * sigmoid_fast(gelu_2z(g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void act_both_fast(float g, float& a, float& slope) {
  if constexpr (ACT == EXTERND_ACT_SILU) {
    const float p = sigmoid_fast(g);
    a = g * p;
    slope = fmaf(a, 1.f - p, p);
  } else if constexpr (ACT == EXTERND_ACT_GELU) {
    const float phi = normal_cdf_fast(g);
    a = g * phi;
    slope = fmaf(0.3989422804014327f * g, __builtin_amdgcn_exp2f(-0.7213475204444817f * g * g), phi);
  } else {
    const float p = sigmoid_fast(gelu_2z(g));
    a = g * p;
    const float q = p * (1.f - p);   // 0 where p is 0 or 1: the cubic may overflow there
    slope = p + (q == 0.f ? 0.f : g * q * gelu_2z_slope(g));
  }
}

}  // namespace externd
