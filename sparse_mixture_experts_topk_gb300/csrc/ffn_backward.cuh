// Shared by the expert FFN's gradient kernels: the activations' slopes.
#pragma once

#include "common.cuh"

namespace moe {

// GELU'(a) = Phi(a) + a phi(a), Phi and phi the normal distribution and density.
__device__ __forceinline__ float gelu_slope(float a) {
  return 0.5f * (1.0f + erff(a * 0.70710678118654752f)) + a * expf(-0.5f * a * a) * 0.39894228040143268f;
}

// h = SiLU(a) u: the gradients of a and u from dh.  SiLU'(a) = s (1 + a (1 - s)), s = sigmoid(a).
__device__ __forceinline__ void swiglu_gradient(float a, float u, float dh, float* da, float* du) {
  const float s = 1.0f / (1.0f + expf(-a));
  *da = dh * u * (s * (1.0f + a * (1.0f - s)));
  *du = dh * (a * s);
}

}  // namespace moe
