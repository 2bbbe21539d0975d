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

// 1 / x to about 2^-23 of itself, 0 for an infinite x (a division that minds results and divisors
// below 2^-126, which do not occur here, takes several times the instructions).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x Sigmoid(x) = x / (1 + e^-x)
__device__ __forceinline__ float silu(float x) {
  return x * rcp(1.f + ex2(-kLog2e * x));
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|, small results to their own last bits:
// log(1 + e) = 2 artanh(r), r = e / (2 + e) <= 1/3, by the series r + r^3 / 3 + ... + r^13 / 13,
// whose rest is below 2^-26 of it.  (log of the rounded 1 + e keeps three digits at v = -9.)
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-kLog2e * fabsf(v));
  const float r = e * rcp(2.f + e), r2 = r * r;
  float p = fmaf(r2, 1.f / 13, 1.f / 11);
  p = fmaf(r2, p, 1.f / 9);
  p = fmaf(r2, p, 1.f / 7);
  p = fmaf(r2, p, 1.f / 5);
  p = fmaf(r2, p, 1.f / 3);
  p = fmaf(r2, p, 1.f);
  return fmaf(2.f * r, p, fmaxf(v, 0.f));
}

// The same of two values at once (packed products: half the instructions).
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 silu2(float2 x) {
  const float2 u = __fmul2_rn(both(-kLog2e), x);
  const float2 q = __fadd2_rn(both(1.f), make_float2(ex2(u.x), ex2(u.y)));
  return __fmul2_rn(x, make_float2(rcp(q.x), rcp(q.y)));
}
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 e = make_float2(ex2(-kLog2e * fabsf(v.x)), ex2(-kLog2e * fabsf(v.y)));
  const float2 q = __fadd2_rn(both(2.f), e);
  const float2 r = __fmul2_rn(e, make_float2(rcp(q.x), rcp(q.y)));
  const float2 r2 = __fmul2_rn(r, r);
  float2 p = __ffma2_rn(r2, both(1.f / 13), both(1.f / 11));
  p = __ffma2_rn(r2, p, both(1.f / 9));
  p = __ffma2_rn(r2, p, both(1.f / 7));
  p = __ffma2_rn(r2, p, both(1.f / 5));
  p = __ffma2_rn(r2, p, both(1.f / 3));
  p = __ffma2_rn(r2, p, both(1.f));
  return __ffma2_rn(__fadd2_rn(r, r), p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

}  // namespace kda
