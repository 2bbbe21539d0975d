// kda_norm_rope.cu -- per-head RMSNorm of q and k and the rotation by position, in
// one pass over both.  Row x of 128 channels (token t, head h), F frequencies f_i:
//     y = w * x / sqrt(mean(x^2) + eps)
//     (a, b) = (y_i, y_{i+F})  or  (y_{2i}, y_{2i+1}),   phi = pos[axis_i][t] * f_i
//     (a, b) <- (a cos phi - b sin phi, a sin phi + b cos phi),  i < F
// and the channels from 2F on pass through.  Everything is fp32 but the angle: at
// position 2^20 an fp32 product is off by 0.06 rad, so it is taken in fp64, reduced to
// a fraction of a turn there, and only the fraction goes to the fp32 sine and cosine.
// One rounding, at the store.
//
// Bound by HBM: a row is read and written once.  A CTA owns whole tokens: its threads
// first put the tokens' F sines and cosines (all heads share them) into shared memory,
// then a half warp per row holds 8 channels a lane (16-byte accesses for bf16), sums
// the squares by a half-warp all-reduce and takes the other half of a pair from the
// lane that holds it by one shuffle.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;  // tokens of one CTA (shared sine/cosine table)
constexpr int kRopeMaxFreq = kD / 2;

// sin and cos of p * f: the turn count in fp64, its fraction in fp32.
__device__ __forceinline__ float2 sincos_turns(int32_t p, float f) {
  double u = (double)p * (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  u -= rint(u);
  float s, c;
  sincospif(2.f * (float)u, &s, &c);
  return make_float2(c, s);
}

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  const float *wq, *wk;       // null: ones
  const int32_t* pos;         // [n_axes][n_tokens]
  const int32_t* axis;        // [F] (null: axis 0)
  const float* freq;          // [F]
  int64_t n_tokens;
  int64_t sq, sk, sqo, sko;   // elements between tokens
  float eps;                  // < 0: no norm
  int n_axes, F, Hq, Hk, tokens;  // tokens: of one CTA
};

template <typename T, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(RopeArgs a, int* err) {
  __shared__ float2 cs[kRopeMaxTokens * kRopeMaxFreq];  // (cos, sin) of (token, frequency)
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.n_tokens - t0);
  for (int e = tid; e < nt * a.F; e += kRopeThreads) {
    const int t = e / a.F, i = e - t * a.F;
    int ax = a.axis ? __ldg(a.axis + i) : 0;
    if (ax < 0 || ax >= a.n_axes) {  // reported; axis 0 keeps the read in bounds
      if (err) atomicExch(err, kDevErrBadAxis);
      ax = 0;
    }
    cs[e] = sincos_turns(__ldg(a.pos + ax * a.n_tokens + t0 + t), __ldg(a.freq + i));
  }
  const int hl = tid & 15;  // lane of the half warp: channels 8 hl .. 8 hl + 7
  float wq[8], wk[8];
  if (kNorm) {
#pragma unroll
    for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.f;
    if (a.wq) load8(a.wq + 8 * hl, wq);
    if (a.wk) load8(a.wk + 8 * hl, wk);
  }
  __syncthreads();
  const int R = a.Hq + a.Hk, rows = nt * R;
  const int F8 = a.F >> 3;  // lanes of one half of the rotated channels (half-split pairs)
  constexpr int kHalfWarps = kRopeThreads / 16, kBatch = 4;
  // every half warp of a warp runs the same number of rounds: the shuffles are uniform
  for (int base = 0; base < rows; base += kHalfWarps * kBatch) {
    float x[kBatch][8];
    int tk[kBatch], hh[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = base + b * kHalfWarps + (tid >> 4);
      tk[b] = row / R;
      hh[b] = row - tk[b] * R;
      if (row < rows) {
        const T* p = hh[b] < a.Hq
                         ? static_cast<const T*>(a.q) + (t0 + tk[b]) * a.sq + hh[b] * kD
                         : static_cast<const T*>(a.k) + (t0 + tk[b]) * a.sk + (hh[b] - a.Hq) * kD;
        load8(p + 8 * hl, x[b]);
      } else {
        tk[b] = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[b][i] = 0.f;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool isq = hh[b] < a.Hq;
      if (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[b][i], x[b][i], ss);
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[b][i] *= r * (isq ? wq[i] : wk[i]);
      }
      const float2* c = cs + max(tk[b], 0) * a.F;
      float y[8];
      if (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = 4 * hl + i;
          const float2 w = f < a.F ? c[f] : make_float2(1.f, 0.f);
          y[2 * i] = x[b][2 * i] * w.x - x[b][2 * i + 1] * w.y;
          y[2 * i + 1] = x[b][2 * i] * w.y + x[b][2 * i + 1] * w.x;
        }
      } else {
        const bool low = hl < F8, rot = hl < 2 * F8;
        // lane of the half warp that holds the other half of this lane's pairs
        const int other = rot ? (low ? hl + F8 : hl - F8) : hl;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = __shfl_sync(0xffffffffu, x[b][i], other, 16);
          const float2 w = rot ? c[8 * (low ? hl : other) + i] : make_float2(1.f, 0.f);
          y[i] = low ? x[b][i] * w.x - z * w.y : x[b][i] * w.x + z * w.y;
          if (!rot) y[i] = x[b][i];
        }
      }
      if (tk[b] >= 0) {
        T* p = isq ? static_cast<T*>(a.qo) + (t0 + tk[b]) * a.sqo + hh[b] * kD
                   : static_cast<T*>(a.ko) + (t0 + tk[b]) * a.sko + (hh[b] - a.Hq) * kD;
        store8(p + 8 * hl, y);
      }
    }
  }
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, bool inter, bool norm, int* err, cudaStream_t s) {
  const int64_t ctas = (a.n_tokens + a.tokens - 1) / a.tokens;
  using Fn = void (*)(RopeArgs, int*);
  static const Fn fn[2][2] = {{norm_rope_kernel<T, false, false>, norm_rope_kernel<T, false, true>},
                              {norm_rope_kernel<T, true, false>, norm_rope_kernel<T, true, true>}};
  fn[inter][norm]<<<(unsigned)ctas, kRopeThreads, 0, s>>>(a, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const void* q, const void* k, int bf16, const float* wq,
                             const float* wk, float eps, const int32_t* pos, int n_axes,
                             const int32_t* axis, const float* freq, int F, int interleaved,
                             void* qo, void* ko, int64_t n_tokens, int Hq, int Hk, int64_t sq,
                             int64_t sk, int64_t sqo, int64_t sko, int* err, cudaStream_t s) {
  RopeArgs a{q, k, qo, ko, wq, wk, pos, axis, freq, n_tokens, sq, sk, sqo, sko, eps, n_axes, F,
             Hq, Hk, 1};
  // about 64 rows a CTA (four a half warp), so that a row's load has others beside it
  a.tokens = 64 / (Hq + Hk);
  a.tokens = a.tokens < 1 ? 1 : (a.tokens > kRopeMaxTokens ? kRopeMaxTokens : a.tokens);
  ProfScope prof_scope("kda_qk_norm_rope", s);
  return bf16 ? launch_rope_t<__nv_bfloat16>(a, interleaved != 0, eps >= 0.f, err, s)
              : launch_rope_t<float>(a, interleaved != 0, eps >= 0.f, err, s);
}

}  // namespace kda
