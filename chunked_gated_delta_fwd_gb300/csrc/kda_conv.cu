// kda_conv.cu -- short causal depthwise convolution over packed sequences, and for new tokens
// with the last inputs kept:
//     y_t[c] = act(bias[c] + sum_{j < W} w[c][j] x_{t-W+1+j}[c]),   W = 2 .. 4,
// act the identity or SiLU; what lies before a sequence comes from its kept inputs (or is 0).
//
// Bound by HBM: x is read and y written once.  A lane holds four channels and
// walks a run of tokens with the last W - 1 inputs in registers, so a run reads W - 1 rows more
// than it has (from L2: its neighbour reads them as well).  Eight rows are on their way while eight
// are worked on, and the eight behind them on theirs to L2 (79 -> 70 us in the first case below);
// products are packed pairs.  Sums are fp32, rounded once.  8192 tokens x 12288
// channels, W = 4 with SiLU: bf16 65 us (6.2 TB/s), fp32 123 us (6.5 TB/s); 512 single tokens of as many
// channels bf16 20 to 21 us (5 TB/s), fp32 33 us (6.1 TB/s): some 6 us a call that do not grow with it,
// the first loads and the last stores; one token 4.4 us cold, 1.5 us behind another call.
#include <algorithm>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_layer_math.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 128;
constexpr int kGroup = 8;      // rows of a lane in flight (prompts)
constexpr int kStepGroup = 4;  // (new tokens)

// Four channels of a row: as they lie in memory, and as pairs of fp32.
template <typename T> struct Words;
template <> struct Words<__nv_bfloat16> { using type = uint2; };
template <> struct Words<float> { using type = uint4; };
template <typename T> using Row = typename Words<T>::type;
constexpr int kVec = 4, kPairs = 2;
__device__ __forceinline__ void unpack(const uint2& u, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4& u, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void pack(const float2 (&f)[2], uint2& u) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0].x, f[0].y), b = __floats2bfloat162_rn(f[1].x, f[1].y);
  u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void pack(const float2 (&f)[2], uint4& u) {
  u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                 __float_as_uint(f[1].y));
}

// The taps of a lane's channels, and one output row from a window of rows, the oldest first.
template <typename T, int kW>
struct Taps {
  float2 w[kW][kPairs], b[kPairs];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int cv) {
    float raw[kVec * kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(weight) + (int64_t)cv * kW + i);
      raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
    }
    const float4 v = bias ? __ldg(reinterpret_cast<const float4*>(bias) + cv)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    b[0] = make_float2(v.x, v.y);
    b[1] = make_float2(v.z, v.w);
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j][i] = make_float2(raw[2 * i * kW + j], raw[(2 * i + 1) * kW + j]);
  }
  template <bool kAct>
  __device__ __forceinline__ Row<T> row(const float2 (*window)[kPairs]) const {
    float2 y[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      y[i] = b[i];
#pragma unroll
      for (int j = 0; j < kW; ++j) y[i] = __ffma2_rn(w[j][i], window[j][i], y[i]);
    }
    if constexpr (kAct) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) y[i] = silu2(y[i]);
    }
    Row<T> u;
    pack(y, u);
    return u;
  }
};

// id / lanes, in 32 bits where they do.
__device__ __forceinline__ int64_t quotient(int64_t id, int lanes) {
  return (id >> 32) != 0 ? id / lanes : (int64_t)((uint32_t)id / (uint32_t)lanes);
}

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
  int N, C, run;
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
  const int lanes = a.C / kVec;
  for (int n = blockIdx.x; n < a.N; n += a.ends) {
    const int64_t b = a.cu ? __ldg(a.cu + n) : 0, e = a.cu ? __ldg(a.cu + n + 1) : 0;
    bad |= b < 0 || e < b || e > a.NT || (n == 0 && b != 0) || (n == a.N - 1 && e != a.NT);
    if (!a.last || b != e) continue;
    const int64_t at = (int64_t)n * K * lanes;
    for (int i = threadIdx.x; i < K * lanes; i += blockDim.x)
      reinterpret_cast<Row<T>*>(a.last)[at + i] =
          a.state ? reinterpret_cast<const Row<T>*>(a.state)[at + i] : Row<T>{};
  }
  if (bad && threadIdx.x == 0 && err) atomicExch(err, kDevErrBadSeqlens);
}

template <typename T, int kW, bool kAct>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvArgs a, int* err) {
  constexpr int K = kW - 1;
  constexpr int kPiece = (int)sizeof(Row<T>);
  if ((int)blockIdx.x < a.ends) {
    conv_ends<T>(a, K, err);
    return;
  }
  const int lanes = a.C / kVec;
  const int64_t id = (int64_t)(blockIdx.x - a.ends) * kConvThreads + threadIdx.x;
  const int64_t tile = quotient(id, lanes);
  const int cv = (int)(id - tile * lanes);
  if (tile >= a.runs) return;
  const char* x = a.x + kPiece * (int64_t)cv;
  char* y = a.y + kPiece * (int64_t)cv;
  // The first rows and the taps are on their way while the run's sequence is looked up.
  const int64_t guess = tile * a.run;
#pragma unroll
  for (int i = -K; i < kGroup; ++i)
    if (guess + i >= 0 && guess + i < a.NT) prefetch(x + (guess + i) * a.sx);
  Taps<T, kW> taps;
  taps.load(a.w, a.b, cv);
  Span sp, after;
  int64_t t = run_begin<kW>(a, guess, sp);
  const int64_t stop = run_begin<kW>(a, min(guess + a.run, a.NT), after);
  if (t >= stop) return;
  const int64_t kept = (int64_t)a.C * sizeof(T);  // bytes of a kept row
  const Row<T> zero{};
  float2 win[K + kGroup][kPairs];
  Row<T> ahead[kGroup];
  const char* xr = nullptr;  // the row that is fetched next
  auto fetch = [&](int left) {
    if (left >= kGroup) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i, xr += a.sx) ahead[i] = *reinterpret_cast<const Row<T>*>(xr);
      if (left >= 2 * kGroup) {
        const char* p = xr;
#pragma unroll
        for (int i = 0; i < kGroup; ++i, p += a.sx) prefetch(p);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kGroup - 1; ++i, xr += a.sx)
        if (i < left) ahead[i] = *reinterpret_cast<const Row<T>*>(xr);
    }
  };
  while (t < stop) {  // sequence by sequence
    const int64_t end = min(sp.end, stop);
    int left = (int)(end - t);  // (a run's tokens at most, and W - 2)
    xr = x + t * a.sx;
    char* yr = y + t * a.sy;
    fetch(left);
    Row<T> old[K];
    if (t == sp.begin) {
      const int64_t at = (int64_t)sp.n * K * kept + kPiece * (int64_t)cv;
#pragma unroll
      for (int r = 0; r < K; ++r)
        old[r] = a.state ? *reinterpret_cast<const Row<T>*>(a.state + at + r * kept) : zero;
      if (a.last) {
        const int64_t len = sp.end - sp.begin;
        Row<T> out[K];
#pragma unroll
        for (int r = 0; r < K; ++r) {
          if (len + r >= K) {
            out[r] = *reinterpret_cast<const Row<T>*>(x + (sp.end - K + r) * a.sx);
          } else {
            out[r] = zero;
#pragma unroll
            for (int m = 0; m < K; ++m)
              if (m == len + r) out[r] = old[m];
          }
        }
#pragma unroll
        for (int r = 0; r < K; ++r) *reinterpret_cast<Row<T>*>(a.last + at + r * kept) = out[r];
      }
    } else {
#pragma unroll
      for (int r = 0; r < K; ++r)  // (all of them, where the offsets are sound)
        old[r] = t - K + r >= sp.begin ? *reinterpret_cast<const Row<T>*>(x + (t - K + r) * a.sx) : zero;
    }
#pragma unroll
    for (int r = 0; r < K; ++r) unpack(old[r], win[r]);
    for (;; left -= kGroup) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) unpack(ahead[i], win[K + i]);
      fetch(left - kGroup);
      if (left < kGroup) break;
#pragma unroll
      for (int i = 0; i < kGroup; ++i, yr += a.sy)
        *reinterpret_cast<Row<T>*>(yr) = taps.template row<kAct>(win + i);
#pragma unroll
      for (int r = 0; r < K; ++r)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) win[r][j] = win[kGroup + r][j];
    }
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i, yr += a.sy)
      if (i < left) *reinterpret_cast<Row<T>*>(yr) = taps.template row<kAct>(win + i);
    t = end;
    if (t < stop) sp = span_of(a, t);
  }
}

// T new tokens of N sequences (kOne: one); the kept inputs end as they are behind the first
// n_advance.  Several sequences a lane, to read the taps once, are slower (512 sequences x 12288
// channels: 39 us with two or four).
template <typename T, int kW, bool kAct, bool kOne>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(
    const ConvArgs a, char* __restrict__ state, const int32_t* __restrict__ n_advance, int T_) {
  constexpr int K = kW - 1, kG = kOne ? 1 : kStepGroup;
  constexpr int kPiece = (int)sizeof(Row<T>);
  const int lanes = a.C / kVec, Tn = kOne ? 1 : T_;
  const int64_t id = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t n = quotient(id, lanes);
  if (n >= a.N) return;
  const int cv = (int)(id - n * lanes);
  const int64_t kept = (int64_t)a.C * sizeof(T);
  char* st = state + n * K * kept + kPiece * (int64_t)cv;
  const char* x = a.x + n * Tn * a.sx + kPiece * (int64_t)cv;
  char* y = a.y ? a.y + n * Tn * a.sy + kPiece * (int64_t)cv : nullptr;
  Row<T> win[K + kG];
#pragma unroll
  for (int r = 0; r < K; ++r) win[r] = *reinterpret_cast<const Row<T>*>(st + r * kept);
#pragma unroll
  for (int i = 0; i < kG; ++i)
    if (i < Tn) win[K + i] = *reinterpret_cast<const Row<T>*>(x + i * a.sx);
  int adv = Tn;
  if (!kOne && n_advance) {
    adv = __ldg(n_advance + n);
    adv = adv < 0 ? 0 : (adv > Tn ? Tn : adv);
  }
  Taps<T, kW> taps;
  if (y) taps.load(a.w, a.b, cv);
  for (int t = 0; t < Tn; t += kG) {
    Row<T> ahead[kG];
    if (!kOne) {
#pragma unroll
      for (int i = 0; i < kG; ++i)
        if (t + kG + i < Tn) ahead[i] = *reinterpret_cast<const Row<T>*>(x + (t + kG + i) * a.sx);
    }
    float2 f[K + kG][kPairs];
    if (y) {
#pragma unroll
      for (int i = 0; i < K + kG; ++i) unpack(win[i], f[i]);
    }
#pragma unroll
    for (int i = 0; i < kG; ++i) {
      if (t + i >= Tn) continue;
      if (y) *reinterpret_cast<Row<T>*>(y + (t + i) * a.sy) = taps.template row<kAct>(f + i);
      if (t + i + 1 == adv) {
#pragma unroll
        for (int r = 0; r < K; ++r) *reinterpret_cast<Row<T>*>(st + r * kept) = win[i + 1 + r];
      }
    }
    if (!kOne) {
#pragma unroll
      for (int r = 0; r < K; ++r) win[r] = win[kG + r];
#pragma unroll
      for (int i = 0; i < kG; ++i) win[K + i] = ahead[i];
    }
  }
}

template <typename F>
void with_width(int W, F f) {
  if (W == 2) f(std::integral_constant<int, 2>{});
  else if (W == 3) f(std::integral_constant<int, 3>{});
  else f(std::integral_constant<int, 4>{});
}

template <typename T>
cudaError_t launch_conv_t(ConvArgs a, int W, int act, int* err, cudaStream_t s) {
  const int lanes = a.C / kVec;
  // Runs as long as they leave some 500 lanes an SM, up to 64 tokens: a lane finds its sequence, its
  // taps and its first rows once a run (8192 tokens x 12288 channels: 96, 83, 81 us in runs of 16, 32
  // and 64).
  a.run = 64;
  while (a.run > kGroup && a.NT * lanes / a.run < 152 * 512) a.run /= 2;
  a.runs = (a.NT + a.run - 1) / a.run;
  const int64_t blocks = (a.runs * lanes + kConvThreads - 1) / kConvThreads;
  // (without offsets there is something to see to only if no sequence has tokens)
  a.ends = a.cu || a.NT == 0 ? std::min(a.N, 152) : 0;
  if (blocks + a.ends > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_conv", s);
  with_width(W, [&](auto w) {
    constexpr int kW = decltype(w)::value;
    const auto fn = act ? conv_kernel<T, kW, true> : conv_kernel<T, kW, false>;
    fn<<<(unsigned)(blocks + a.ends), kConvThreads, 0, s>>>(a, err);
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
             sx * e, sy * e, 0, n_seqs, C, 0, 0};
  return bf16 ? launch_conv_t<__nv_bfloat16>(a, W, act, err, s)
              : launch_conv_t<float>(a, W, act, err, s);
}

cudaError_t launch_conv_step(const void* x, int bf16, const float* w, const float* b, void* state,
                             void* y, const int32_t* n_advance, int N, int T, int C, int W,
                             int64_t sx, int64_t sy, int act, cudaStream_t s) {
  const int e = bf16 ? 2 : 4;
  ConvArgs a{static_cast<const char*>(x), static_cast<char*>(y), w, b, nullptr, nullptr, nullptr, T,
             (int64_t)N * T, sx * e, sy * e, 0, N, C, 0, 0};
  const int64_t lanes = C / kVec;
  const int64_t blocks = (N * lanes + kConvThreads - 1) / kConvThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_conv_step", s);
  const bool one = T == 1 && !n_advance && y;
  with_width(W, [&](auto w_) {
    constexpr int kW = decltype(w_)::value;
    auto pick = [&](auto act_, auto one_) {
      constexpr bool kAct = decltype(act_)::value, kOne = decltype(one_)::value;
      return bf16 ? conv_step_kernel<__nv_bfloat16, kW, kAct, kOne>
                  : conv_step_kernel<float, kW, kAct, kOne>;
    };
    const std::true_type yes;
    const std::false_type no;
    const auto fn = act ? (one ? pick(yes, yes) : pick(yes, no)) : (one ? pick(no, yes) : pick(no, no));
    fn<<<(unsigned)blocks, kConvThreads, 0, s>>>(a, static_cast<char*>(state), n_advance, T);
  });
  return cudaGetLastError();
}

}  // namespace kda
