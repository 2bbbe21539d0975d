// kda_scan_step.cu -- new tokens of the selective state space scan, the states of N sequences
// updated in place (T <= 16 tokens a sequence, the state kept as it is behind the first
// n_advance, the outputs of all T written):
//     h <- exp(delta_t A) h + delta_t x_t B_t,   y_t = (C_t . h + D x_t) SiLU(z_t)
//
// Bound by HBM: 8 bytes a state and call.  A lane holds four states of a channel (16-byte
// accesses, a warp's are contiguous); S / 4 lanes share a channel.
#include "kda_internal.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 128;

template <typename T, int kS>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(
    const ScanArgs a, float* __restrict__ state, const int32_t* __restrict__ n_advance) {
  constexpr int kLn = kS / 4;
  const int64_t id = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  const int64_t ch = id / kLn;  // n * C + c
  const int sub = (int)(id % kLn);
  const bool on = ch < (int64_t)a.N * a.C;
  const int64_t n = on ? ch / a.C : 0;
  const int c = on ? (int)(ch - n * a.C) : 0;
  const int Tn = (int)a.T;
  int adv = Tn;
  if (n_advance) {
    adv = __ldg(n_advance + n);
    adv = adv < 0 ? 0 : (adv > Tn ? Tn : adv);
  }
  const int g = c / (a.C / a.G);
  float4* at = reinterpret_cast<float4*>(state) + (n * a.C + c) * kLn + sub;
  float h[4], A[4];
  load4(reinterpret_cast<const float*>(at), h);
  load4(a.A + (int64_t)c * kS + 4 * sub, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
  const float bias = a.bias ? __ldg(a.bias + c) : 0.f, skip = a.D ? __ldg(a.D + c) : 0.f;
  for (int t = 0; t < Tn; ++t) {
    const int64_t row = n * Tn + t;
    const float xv = to_f32(static_cast<const T*>(a.x)[row * a.sx + c]);
    float d = to_f32(static_cast<const T*>(a.dt)[row * a.sdt + c]) + bias;
    if (a.softplus) d = softplus(d);
    float b[4], cc[4];
    load4(static_cast<const T*>(a.B) + row * a.sB + g * kS + 4 * sub, b);
    load4(static_cast<const T*>(a.Cm) + row * a.sC + g * kS + 4 * sub, cc);
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(ex2(d * A[i]), h[i], d * xv * b[i]);
      acc = fmaf(cc[i], h[i], acc);
    }
    if (on && t + 1 == adv) *at = make_float4(h[0], h[1], h[2], h[3]);
    if (!a.y) continue;
#pragma unroll
    for (int m = 1; m < kLn; m *= 2) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    acc = fmaf(skip, xv, acc);
    if (a.z) acc *= silu(to_f32(static_cast<const T*>(a.z)[row * a.sz + c]));
    if (on && sub == 0) static_cast<T*>(a.y)[row * a.sy + c] = from_f32<T>(acc);
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs& a, int bf16, int S, float* state,
                             const int32_t* n_advance, bool multi, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.N * a.C * (S / 4) + kStepThreads - 1) / kStepThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope(multi ? "kda_scan_multi_step" : "kda_scan_step", s);
  with_states(S, [&](auto k) {
    constexpr int kS = decltype(k)::value;
    if (bf16)
      scan_step_kernel<__nv_bfloat16, kS><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, state, n_advance);
    else
      scan_step_kernel<float, kS><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, state, n_advance);
  });
  return cudaGetLastError();
}

}  // namespace kda
