// Shared by the expert FFN's gradient kernels: the activations' slopes.
#pragma once

#include "common.cuh"

namespace moe {

// GELU'(a) = Phi(a) + a phi(a), Phi and phi the normal distribution and density.
__device__ __forceinline__ float gelu_slope(float a) {
  return 0.5f * (1.0f + erff(a * 0.70710678118654752f)) + a * expf(-0.5f * a * a) * 0.39894228040143268f;
}

// The same from one exponential, for the tensor-core kernels, whose epilogue
// the erf above would bound: Phi(|a|) = 1 - phi(a) (c1 t + .. + c5 t^5) with
// t = 1 / (1 + 0.2316419 |a|), Abramowitz and Stegun, Handbook of Mathematical
// Functions, 26.2.17 (absolute error below 7.5e-8, an fp32 rounding of 1).
// CUDA bounds the error of __expf(-z) by 2 + 1.2 z units of the last place; with
// z = a^2 / 2 that adds at most 1.3e-7 to the slope, whatever a is.
__device__ __forceinline__ float gelu_slope_fast(float a) {
  const float x = fabsf(a);
  const float t = __fdividef(1.0f, fmaf(0.2316419f, x, 1.0f));
  const float phi = 0.39894228040143268f * __expf(-0.5f * a * a);
  float p = fmaf(1.330274429f, t, -1.821255978f);
  p = fmaf(p, t, 1.781477937f);
  p = fmaf(p, t, -0.356563782f);
  p = fmaf(p, t, 0.319381530f) * t;
  const float upper = phi * p;                       // 1 - Phi(|a|)
  return fmaf(a, phi, a >= 0.0f ? 1.0f - upper : upper);
}

// h = SiLU(a) u: the gradients of a and u from dh.  SiLU'(a) = s (1 + a (1 - s)),
// s = sigmoid(a) = 1 / (1 + exp(-a)), which overflow takes to its limit 0.
__device__ __forceinline__ void swiglu_slopes(float s, float a, float u, float dh, float* da, float* du) {
  *da = dh * u * (s * (1.0f + a * (1.0f - s)));
  *du = dh * (a * s);
}
__device__ __forceinline__ void swiglu_gradient(float a, float u, float dh, float* da, float* du) {
  swiglu_slopes(1.0f / (1.0f + expf(-a)), a, u, dh, da, du);
}
// With the special-function unit's exponential and quotient.  CUDA bounds the
// exponential's error by 2 + 1.2 |a| units of the last place, the quotient's by
// 2.  s takes the exponential's times 1 - s: below 3e-7 in size anywhere, and
// relative to s at most 1.3e-5 (a = -87, where s is 1e-38).  A rounding of
// the result to bf16 is 2e-3.
__device__ __forceinline__ void swiglu_gradient_fast(float a, float u, float dh, float* da, float* du) {
  swiglu_slopes(__fdividef(1.0f, 1.0f + __expf(-a)), a, u, dh, da, du);
}

}  // namespace moe
