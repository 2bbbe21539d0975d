// kda_scan.cu -- selective state space scan over packed sequences: for every channel c with
// states s = 0 .. S-1 (S = 8, 16, 32) and delta_t = softplus(dt_t + bias),
//     h_t[s] = exp(delta_t A[s]) h_{t-1}[s] + delta_t x_t B_t[s]
//     y_t    = (sum_s C_t[s] h_t[s] + D x_t) SiLU(z_t)
// B and C are shared by the channels of a group.  The states are fp32.
//
// A lane holds eight states of one channel and walks the tokens; S / 8 lanes share a channel.
#include <algorithm>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename T, int kS>
__global__ void __launch_bounds__(32) scan_kernel(const ScanArgs a, int* err) {
  constexpr int kLn = kS / 8, kCh = 32 / kLn;
  const int lane = threadIdx.x;
  const int per_group = a.C / a.G;
  const int blocks = (per_group + kCh - 1) / kCh;  // of a group
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / ((int64_t)blocks * a.G));
  const int rest = (int)(unit - (int64_t)n * blocks * a.G);
  const int g = rest / blocks, in = (rest - g * blocks) * kCh + lane / kLn;
  int64_t t0, t1;
  if (!seq_range(a, n, t0, t1) && threadIdx.x == 0 && err) atomicExch(err, kDevErrBadSeqlens);
  const bool on = in < per_group;
  const int c = g * per_group + (on ? in : 0), s0 = 8 * (lane % kLn);
  const T* x = static_cast<const T*>(a.x) + c;
  const T* dt = static_cast<const T*>(a.dt) + c;
  const T* z = a.z ? static_cast<const T*>(a.z) + c : nullptr;
  const T* B = static_cast<const T*>(a.B) + g * kS + s0;
  const T* Cm = static_cast<const T*>(a.Cm) + g * kS + s0;
  T* y = static_cast<T*>(a.y) + c;
  const float bias = a.bias ? a.bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
  float A[8], h[8];
  load8(a.A + (int64_t)c * kS + s0, A);
#pragma unroll
  for (int i = 0; i < 8; ++i) A[i] *= kLog2e;
  const int64_t at = ((int64_t)n * a.C + c) * kS + s0;
  if (a.h0) {
    load8(a.h0 + at, h);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0.f;
  }
  for (int64_t t = t0; t < t1; ++t) {
    const float xv = to_f32(x[t * a.sx]);
    float d = to_f32(dt[t * a.sdt]) + bias;
    if (a.softplus) d = softplus(d);
    float b[8], cc[8];
    load8(B + t * a.sB, b);
    load8(Cm + t * a.sC, cc);
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = fmaf(ex2(d * A[i]), h[i], d * xv * b[i]);
      acc = fmaf(cc[i], h[i], acc);
    }
#pragma unroll
    for (int m = 1; m < kLn; m *= 2) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    acc = fmaf(skip, xv, acc);
    if (z) acc *= silu(to_f32(z[t * a.sz]));
    if (on && s0 == 0) y[t * a.sy] = from_f32<T>(acc);
  }
  if (a.hT && on) store8(a.hT + at, h);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, int bf16, int S, int* err, cudaStream_t s) {
  const int ch = 256 / S;
  const int64_t units = (int64_t)a.N * a.G * ((a.C / a.G + ch - 1) / ch);
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_scan", s);
  with_states(S, [&](auto k) {
    constexpr int kS = decltype(k)::value;
    if (bf16)
      scan_kernel<__nv_bfloat16, kS><<<(unsigned)units, 32, 0, s>>>(a, err);
    else
      scan_kernel<float, kS><<<(unsigned)units, 32, 0, s>>>(a, err);
  });
  return cudaGetLastError();
}

}  // namespace kda
