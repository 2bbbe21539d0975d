// kda_conv.cu -- short causal depthwise convolution over packed sequences, and for new tokens
// with the last inputs kept:
//     y_t[c] = act(bias[c] + sum_{j < W} w[c][j] x_{t-W+1+j}[c]),   W = 2 .. 4,
// act the identity or SiLU; what lies before a sequence comes from its kept inputs (or is 0).
//
// Bound by HBM: x is read and y written once.  A lane holds 16 bytes of channels of a row and
// walks a run of tokens with the last W - 1 inputs in registers, so a run reads W - 1 rows more
// than it has (from L2: its neighbour reads them as well).  Sums are fp32, rounded once.
#include <algorithm>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_layer_math.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 128;
constexpr int kGroup = 4;  // rows of a lane in flight

// 16 bytes of channels: their count, and as fp32.
template <typename T> struct Vec { static constexpr int n = 16 / (int)sizeof(T); };
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// The taps of a lane's channels, and one output row from the window's rows old .. new.
template <typename T, int kW>
struct Taps {
  static constexpr int n = Vec<T>::n;
  float w[n][kW], b[n];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int c) {
    float raw[n * kW];
#pragma unroll
    for (int i = 0; i < n * kW / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(weight + (int64_t)c * kW) + i);
      raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
#pragma unroll
      for (int j = 0; j < kW; ++j) w[i][j] = raw[i * kW + j];
      b[i] = bias ? __ldg(bias + c + i) : 0.f;
    }
  }
  __device__ __forceinline__ uint4 row(const uint4* window, bool act) const {
    float y[n];
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] = b[i];
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      float f[n];
      unpack(window[j], f);
#pragma unroll
      for (int i = 0; i < n; ++i) y[i] = fmaf(w[i][j], f[i], y[i]);
    }
    if (act) {
#pragma unroll
      for (int i = 0; i < n; ++i) y[i] = silu(y[i]);
    }
    return pack(y);
  }
};

struct ConvArgs {
  const char* x;
  char* y;
  const float *w, *b;
  const char* state;    // [N][W-1][C] (null: zeros)
  char* last;           // [N][W-1][C] (null: not written); may be `state`
  const int32_t* cu;    // [N+1], or null: T_per_seq tokens a sequence
  int64_t T_per_seq, NT;
  int64_t sx, sy;       // bytes between tokens
  int64_t runs;
  int N, C, run, act;
  int ends;  // blocks that look after the sequences as a whole
};

struct Span {
  int64_t begin, end;
  int n;
};

// The sequence that token t belongs to.  Offsets that do not run from 0 to NT upwards give some
// span around t within [0, NT]; conv_ends reports them.
__device__ __forceinline__ Span span_of(const ConvArgs& a, int64_t t) {
  if (!a.cu) {
    const int64_t n = t / a.T_per_seq;
    return {n * a.T_per_seq, (n + 1) * a.T_per_seq, (int)n};
  }
  int lo = 0, hi = a.N - 1;  // the last sequence that begins at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int64_t b = __ldg(a.cu + lo), e = __ldg(a.cu + lo + 1);
  return {max((int64_t)0, min(b, t)), min(a.NT, max(e, t + 1)), lo};
}

// Where the run that would begin at token t begins: the first W - 1 tokens of a sequence stay
// with its first, so that one thread alone reads a sequence's kept inputs (and may overwrite
// them with the new ones).
template <int kW>
__device__ __forceinline__ int64_t run_begin(const ConvArgs& a, int64_t t, Span& sp) {
  if (t >= a.NT) return a.NT;
  sp = span_of(a, t);
  if (t == sp.begin || t - sp.begin >= kW - 1) return t;
  t = min(sp.begin + kW - 1, sp.end);
  if (t == sp.end && t < a.NT) sp = span_of(a, t);
  return t;
}

// Kept inputs of sequences without tokens, and the check of the offsets: the grid's first blocks.
template <typename T>
__device__ void conv_ends(const ConvArgs& a, int K, int* err) {
  bool bad = false;
  const int lanes = a.C / Vec<T>::n;
  for (int n = blockIdx.x; n < a.N; n += a.ends) {
    const int64_t b = a.cu ? __ldg(a.cu + n) : 0, e = a.cu ? __ldg(a.cu + n + 1) : 0;
    bad |= b < 0 || e < b || e > a.NT || (n == 0 && b != 0) || (n == a.N - 1 && e != a.NT);
    if (!a.last || b != e) continue;
    const int64_t at = (int64_t)n * K * lanes;
    for (int i = threadIdx.x; i < K * lanes; i += blockDim.x)
      reinterpret_cast<uint4*>(a.last)[at + i] =
          a.state ? reinterpret_cast<const uint4*>(a.state)[at + i] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (bad && threadIdx.x == 0 && err) atomicExch(err, kDevErrBadSeqlens);
}

template <typename T, int kW>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvArgs a, int* err) {
  constexpr int kV = Vec<T>::n, K = kW - 1;
  if ((int)blockIdx.x < a.ends) {
    conv_ends<T>(a, K, err);
    return;
  }
  const int lanes = a.C / kV;
  const int64_t id = (int64_t)(blockIdx.x - a.ends) * kConvThreads + threadIdx.x;
  const int64_t tile = id / lanes;
  if (tile >= a.runs) return;
  const int cv = (int)(id - tile * lanes);
  Span sp, after;
  int64_t t = run_begin<kW>(a, tile * a.run, sp);
  const int64_t stop = run_begin<kW>(a, min((tile + 1) * a.run, a.NT), after);
  if (t >= stop) return;
  Taps<T, kW> taps;
  taps.load(a.w, a.b, cv * kV);
  const char* x = a.x + 16 * (int64_t)cv;
  char* y = a.y + 16 * (int64_t)cv;
  const int64_t kept = (int64_t)a.C * sizeof(T);  // bytes of a kept row
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 win[K + kGroup];
  while (t < stop) {  // sequence by sequence
    const int64_t end = min(sp.end, stop);
    if (t == sp.begin) {
      const int64_t at = (int64_t)sp.n * K * kept + 16 * (int64_t)cv;
#pragma unroll
      for (int r = 0; r < K; ++r)
        win[r] = a.state ? *reinterpret_cast<const uint4*>(a.state + at + r * kept) : zero;
      if (a.last) {
        const int64_t len = sp.end - sp.begin;
        uint4 out[K];
#pragma unroll
        for (int r = 0; r < K; ++r) {
          if (len + r >= K) {
            out[r] = *reinterpret_cast<const uint4*>(x + (sp.end - K + r) * a.sx);
          } else {
            out[r] = zero;
#pragma unroll
            for (int m = 0; m < K; ++m)
              if (m == len + r) out[r] = win[m];
          }
        }
#pragma unroll
        for (int r = 0; r < K; ++r) *reinterpret_cast<uint4*>(a.last + at + r * kept) = out[r];
      }
    } else {
#pragma unroll
      for (int r = 0; r < K; ++r)  // (all of them, where the offsets are sound)
        win[r] = t - K + r >= sp.begin ? *reinterpret_cast<const uint4*>(x + (t - K + r) * a.sx) : zero;
    }
    while (t < end) {
      const int64_t left = end - t;
      const int m = left < kGroup ? (int)left : kGroup;
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (i < m) win[K + i] = *reinterpret_cast<const uint4*>(x + (t + i) * a.sx);
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (i < m) *reinterpret_cast<uint4*>(y + (t + i) * a.sy) = taps.row(win + i, a.act);
      t += m;
      if (t < end) {  // a whole group
#pragma unroll
        for (int r = 0; r < K; ++r) win[r] = win[kGroup + r];
      }
    }
    if (t < stop) sp = span_of(a, t);
  }
}

// T new tokens of N sequences; the kept inputs end as they are behind the first n_advance.
template <typename T, int kW>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(
    const ConvArgs a, char* __restrict__ state, const int32_t* __restrict__ n_advance, int Tn) {
  constexpr int kV = Vec<T>::n, K = kW - 1;
  const int lanes = a.C / kV;
  const int64_t id = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t n = id / lanes;
  if (n >= a.N) return;
  const int cv = (int)(id - n * lanes);
  int adv = Tn;
  if (n_advance) {
    adv = __ldg(n_advance + n);
    adv = adv < 0 ? 0 : (adv > Tn ? Tn : adv);
  }
  const char* x = a.x + n * Tn * a.sx + 16 * (int64_t)cv;
  char* y = a.y ? a.y + n * Tn * a.sy + 16 * (int64_t)cv : nullptr;
  const int64_t kept = (int64_t)a.C * sizeof(T), at = n * K * kept + 16 * (int64_t)cv;
  uint4 win[K + kGroup];
#pragma unroll
  for (int r = 0; r < K; ++r) win[r] = *reinterpret_cast<const uint4*>(state + at + r * kept);
  Taps<T, kW> taps;
  if (y) taps.load(a.w, a.b, cv * kV);
  for (int t = 0; t < Tn; t += kGroup) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (t + i < Tn) win[K + i] = *reinterpret_cast<const uint4*>(x + (t + i) * a.sx);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (t + i >= Tn) continue;
      if (y) *reinterpret_cast<uint4*>(y + (t + i) * a.sy) = taps.row(win + i, a.act);
      if (t + i + 1 == adv) {
#pragma unroll
        for (int r = 0; r < K; ++r)
          *reinterpret_cast<uint4*>(state + at + r * kept) = win[i + 1 + r];
      }
    }
#pragma unroll
    for (int r = 0; r < K; ++r) win[r] = win[kGroup + r];
  }
}

template <typename F>
void with_width(int W, F f) {
  if (W == 2) f(std::integral_constant<int, 2>{});
  else if (W == 3) f(std::integral_constant<int, 3>{});
  else f(std::integral_constant<int, 4>{});
}

template <typename T>
cudaError_t launch_conv_t(ConvArgs a, int W, int* err, cudaStream_t s) {
  const int lanes = a.C / Vec<T>::n;
  a.run = 16;
  a.runs = (a.NT + a.run - 1) / a.run;
  const int64_t blocks = (a.runs * lanes + kConvThreads - 1) / kConvThreads;
  // (without offsets there is something to see to only if no sequence has tokens)
  a.ends = a.cu || a.NT == 0 ? std::min(a.N, 152) : 0;
  if (blocks + a.ends > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_conv", s);
  with_width(W, [&](auto w) {
    conv_kernel<T, decltype(w)::value><<<(unsigned)(blocks + a.ends), kConvThreads, 0, s>>>(a, err);
  });
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv(const void* x, int bf16, const float* w, const float* b, const void* state,
                        const int32_t* cu, int64_t T_per_seq, void* y, void* last, int64_t n_tokens,
                        int n_seqs, int C, int W, int64_t sx, int64_t sy, int act, int* err,
                        cudaStream_t s) {
  const int e = bf16 ? 2 : 4;
  ConvArgs a{static_cast<const char*>(x), static_cast<char*>(y), w, b,
             static_cast<const char*>(state), static_cast<char*>(last), cu, T_per_seq, n_tokens,
             sx * e, sy * e, 0, n_seqs, C, 0, act, 0};
  return bf16 ? launch_conv_t<__nv_bfloat16>(a, W, err, s) : launch_conv_t<float>(a, W, err, s);
}

cudaError_t launch_conv_step(const void* x, int bf16, const float* w, const float* b, void* state,
                             void* y, const int32_t* n_advance, int N, int T, int C, int W,
                             int64_t sx, int64_t sy, int act, cudaStream_t s) {
  const int e = bf16 ? 2 : 4;
  ConvArgs a{static_cast<const char*>(x), static_cast<char*>(y), w, b, nullptr, nullptr, nullptr, T,
             (int64_t)N * T, sx * e, sy * e, 0, N, C, 0, act, 0};
  const int64_t blocks = ((int64_t)N * (C * e / 16) + kConvThreads - 1) / kConvThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_conv_step", s);
  with_width(W, [&](auto w_) {
    constexpr int kW = decltype(w_)::value;
    if (bf16)
      conv_step_kernel<__nv_bfloat16, kW><<<(unsigned)blocks, kConvThreads, 0, s>>>(
          a, static_cast<char*>(state), n_advance, T);
    else
      conv_step_kernel<float, kW><<<(unsigned)blocks, kConvThreads, 0, s>>>(
          a, static_cast<char*>(state), n_advance, T);
  });
  return cudaGetLastError();
}

}  // namespace kda
