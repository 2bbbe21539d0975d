// kda_layer_math.cuh -- scalar functions of the layers around the recurrences, in fp32.
#pragma once

#include <cuda_runtime.h>

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, off by about 2^-22 of itself; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x Sigmoid(x) = x / (1 + e^-x)
__device__ __forceinline__ float silu(float x) {
  return __fdividef(x, 1.f + ex2(-kLog2e * x));
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|, small results to their own last bits:
// log(1 + e) = 2 artanh(r), r = e / (2 + e) <= 1/3, by the series r + r^3 / 3 + ... + r^13 / 13,
// whose rest is below 2^-26 of it.  (log of the rounded 1 + e keeps three digits at v = -9.)
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-kLog2e * fabsf(v));
  const float r = __fdividef(e, 2.f + e), r2 = r * r;
  float p = fmaf(r2, 1.f / 13, 1.f / 11);
  p = fmaf(r2, p, 1.f / 9);
  p = fmaf(r2, p, 1.f / 7);
  p = fmaf(r2, p, 1.f / 5);
  p = fmaf(r2, p, 1.f / 3);
  p = fmaf(r2, p, 1.f);
  return fmaf(2.f * r, p, fmaxf(v, 0.f));
}

}  // namespace kda
