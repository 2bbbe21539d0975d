// kda_scan_step.cu -- new tokens of the selective state space scan, the states of N sequences
// updated in place (T <= 16 tokens a sequence, the state kept as it is behind the first
// n_advance, the outputs of all T written):
//     h <- exp(delta_t A) h + delta_t x_t B_t,   y_t = (C_t . h + D x_t) SiLU(z_t)
//
// Bound by HBM: 8 bytes a state and call.  A lane holds eight states of a channel (two 16-byte
// accesses, S / 8 lanes side by side in each) of S / 8 sequences at once, and S / 8 lanes share a
// channel: each of them looks after one of the sequences (its step, its gate, its output, once a token
// and channel), and the others get the step by a shuffle.  B and C of the sequences' tokens sit in
// shared memory.  512 sequences x 8192 channels of 16 states, one token: 86 to 91 us, 6.3 TB/s (195 us
// with one sequence a lane, whose lanes each formed the step; 97 with four states a lane and four
// sequences; 118 with sixteen and 114 with two channels of one sequence a lane, whose accesses reach
// into more lines at once); 5 tokens of 96 x 4096: 21 to 24 us (24 to 28 with four states a lane), where
// the tokens (2.6 us each, 3.1) bound it, by what the schedulers can issue.
#include "kda_internal.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 128;

template <typename T, int kS, bool kMulti>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(
    const ScanArgs a, float* __restrict__ state, const int32_t* __restrict__ n_advance) {
  constexpr int kQ = 2, kLn = kS / 4 / kQ, kSlots = kLn, kT = kMulti ? 16 : 1;
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ __align__(16) float BC[2][kSlots * kT][kS];  // rows as in memory: Tn a sequence
  const int Tn = kMulti ? (int)a.T : 1;
  const int per_group = a.C / a.G;
  const int blocks = (per_group * kLn + kStepThreads - 1) / kStepThreads;  // of a group
  const int row_blocks = blocks * a.G;  // (the grid is a multiple of it)
  const int bunch = (int)blockIdx.x / row_blocks;
  const int block = (int)blockIdx.x - bunch * row_blocks, g = block / blocks;
  const int id = (block - g * blocks) * kStepThreads + threadIdx.x;
  const bool on = id < per_group * kLn;
  const int c = g * per_group + (on ? id / kLn : 0), sub = id % kLn;
  const int64_t n0 = (int64_t)bunch * kSlots;
  const int there = (int)min((int64_t)kSlots, a.N - n0);  // sequences
  const bool mine = on && sub < there;
  const int64_t n = n0 + (sub < there ? sub : 0);  // the sequence the lane looks after

  float4* at = reinterpret_cast<float4*>(state) + (n0 * a.C + c) * (kS / 4) + sub;
  const int64_t hop = (int64_t)a.C * (kS / 4);
  float h[kSlots][kQ][4];
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
#pragma unroll
    for (int j = 0; j < kQ; ++j) {
      const float4 v = on && i < there ? __ldcs(at + i * hop + j * kLn) : make_float4(0.f, 0.f, 0.f, 0.f);
      h[i][j][0] = v.x; h[i][j][1] = v.y; h[i][j][2] = v.z; h[i][j][3] = v.w;
    }
  const T* xp = static_cast<const T*>(a.x) + n * Tn * a.sx + c;
  const T* dp = static_cast<const T*>(a.dt) + n * Tn * a.sdt + c;
  const T* zp = a.z ? static_cast<const T*>(a.z) + n * Tn * a.sz + c : nullptr;
  T* yp = a.y ? static_cast<T*>(a.y) + n * Tn * a.sy + c : nullptr;
  T rx, rd, rz;
  auto fetch = [&] {
    rx = *xp;
    rd = *dp;
    if (zp) rz = *zp;
  };
  fetch();
  for (int e = threadIdx.x; e < 2 * there * Tn * (kS / 4); e += kStepThreads) {
    const int q = 4 * (e % (kS / 4)), which = e / (kS / 4) % 2, r = e / (kS / 2);
    const T* src = which ? static_cast<const T*>(a.Cm) + (n0 * Tn + r) * a.sC
                         : static_cast<const T*>(a.B) + (n0 * Tn + r) * a.sB;
    float v[4];
    load4(src + g * kS + q, v);
    store4(&BC[which][r][q], v);
  }
  float A[kQ][4];
#pragma unroll
  for (int j = 0; j < kQ; ++j) {
    load4(a.A + (int64_t)c * kS + 4 * (sub + kLn * j), A[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) A[j][i] *= kLog2e;
  }
  const float bias = a.bias ? __ldg(a.bias + c) : 0.f, skip = a.D ? __ldg(a.D + c) : 0.f;
  int adv = Tn;
  if (kMulti && n_advance) {
    adv = __ldg(n_advance + n);
    adv = adv < 0 ? 0 : (adv > Tn ? Tn : adv);
  }
  int stop[kSlots];  // the tokens behind which the states are stored (0: none)
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int upto = kMulti ? __shfl_sync(kAll, adv, i, kLn) : 1;
    stop[i] = on && i < there ? upto : 0;
  }
  __syncthreads();
#pragma unroll 1
  for (int t = 0; t < Tn; ++t) {
    const float x = to_f32(rx), z = zp ? to_f32(rz) : 0.f;
    float d = to_f32(rd) + bias;
    if (kMulti && t + 1 < Tn) {
      xp += a.sx;
      dp += a.sdt;
      zp += zp ? a.sz : 0;
      fetch();
    }
    if (a.softplus) d = softplus(d);
    const float dx = d * x;
    float acc[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const float di = __shfl_sync(kAll, d, i, kLn), dxi = __shfl_sync(kAll, dx, i, kLn);
      acc[i] = 0.f;
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const int q = 4 * (sub + kLn * j);
        const float4 b = *reinterpret_cast<const float4*>(&BC[0][i * Tn + t][q]);
        const float4 k = *reinterpret_cast<const float4*>(&BC[1][i * Tn + t][q]);
        float (&s)[4] = h[i][j];
        s[0] = fmaf(ex2(di * A[j][0]), s[0], dxi * b.x);
        s[1] = fmaf(ex2(di * A[j][1]), s[1], dxi * b.y);
        s[2] = fmaf(ex2(di * A[j][2]), s[2], dxi * b.z);
        s[3] = fmaf(ex2(di * A[j][3]), s[3], dxi * b.w);
        acc[i] = fmaf(k.x, s[0], fmaf(k.y, s[1], fmaf(k.z, s[2], fmaf(k.w, s[3], acc[i]))));
        if (t + 1 == stop[i]) __stcs(at + i * hop + j * kLn, make_float4(s[0], s[1], s[2], s[3]));
      }
    }
    if (!yp) continue;
    // halving exchange inside a channel's lanes: lane sub ends with sequence sub
#pragma unroll
    for (int m = kLn / 2; m > 0; m /= 2) {
      const bool upper = (sub & m) != 0;
#pragma unroll
      for (int j = 0; j < m; ++j) {
        const float other = __shfl_xor_sync(kAll, upper ? acc[j] : acc[j + m], m);
        acc[j] = (upper ? acc[j + m] : acc[j]) + other;
      }
    }
    float y = fmaf(skip, x, acc[0]);
    if (zp) y *= silu(z);
    if (mine) *yp = from_f32<T>(y);
    yp += a.sy;
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs& a, int bf16, int S, float* state,
                             const int32_t* n_advance, bool multi, cudaStream_t s) {
  const int lanes = S / 8;
  const int64_t blocks = (int64_t)a.G * (((int64_t)a.C / a.G * lanes + kStepThreads - 1) / kStepThreads);
  const int64_t grid = blocks * (((int64_t)a.N + lanes - 1) / lanes);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope(multi ? "kda_scan_multi_step" : "kda_scan_step", s);
  with_states(S, [&](auto k) {
    constexpr int kS = decltype(k)::value;
    using H = __nv_bfloat16;
    const auto fn = multi ? (bf16 ? scan_step_kernel<H, kS, true> : scan_step_kernel<float, kS, true>)
                          : (bf16 ? scan_step_kernel<H, kS, false> : scan_step_kernel<float, kS, false>);
    fn<<<(unsigned)grid, kStepThreads, 0, s>>>(a, state, n_advance);
  });
  return cudaGetLastError();
}

}  // namespace kda
