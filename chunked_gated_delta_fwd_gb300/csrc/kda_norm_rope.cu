// kda_norm_rope.cu -- per-head RMSNorm of q and k and the rotation by position, in
// one pass over both.  Row x of 128 channels (token t, head h), F frequencies f_i:
//     y = w * x / sqrt(mean(x^2) + eps)
//     (a, b) = (y_i, y_{i+F})  or  (y_{2i}, y_{2i+1}),   phi = pos[axis_i][t] * f_i
//     (a, b) <- (a cos phi - b sin phi, a sin phi + b cos phi),  i < F
// and the channels from 2F on pass through.  Everything is fp32 but the angle: at
// position 2^20 an fp32 product is off by 0.06 rad.  A CTA takes every f_i / (2 pi) once, in
// fp64, as a 64-bit fraction of a turn; position times fraction modulo 2^64 is then the
// fraction of a turn of phi, whole turns gone, off by |pos| (2^-63 + |f_i| 2^-107).  (An fp64
// product and reduction for each angle instead: 39.5 us in the 40-head case below against 37.5,
// both replayed from a graph; fp64 has a few lanes an SM.)  One rounding, at the store.
//
// With r = 1 / sqrt(mean(x^2) + eps) a channel's result is r (x_i A_i + x_p B_i), x_p the
// other channel of its pair, A_i = w_i cos phi and B_i = -+ w_p sin phi: the same for all
// heads of a token.  So a warp takes sixteen (fp32: eight) rows, heads of one token where there
// are as many, builds its lanes' A and B once a token and then needs two multiplications a
// channel; the pair's other channel travels as raw input, four shuffles a bf16 row.
//
// Bound by HBM: a row is read and written once (8192 tokens x 192 heads bf16: 127 us, 6.3 TB/s;
// 10007 tokens of 40 heads out of a packed projection: 39 us, 5.3 TB/s; 65536 tokens of 1 + 1
// heads 30 us, 2.3 TB/s: there the angles, 64 for two rows, bound it; fp32, twice the bytes: 281 us,
// 5.7 TB/s, and 76 us, 5.4 TB/s, in the first two cases).  A half warp holds
// a row, 8 channels a lane (16-byte accesses), 128 bytes of a lane in flight.  The CTAs stay
// resident and walk the tokens; the next tokens' sines and cosines (shared by all heads) are formed
// between two barriers' worth of rows.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeCtas = 3;        // resident CTAs an SM
// Rows of a half warp in one unit of its warp, 128 bytes a lane.  kHeads of them belong to one
// token: twice the rows (both half warps share a token, every other head each) or fewer (a half
// warp walks tokens of its own), so that few heads fill a unit too.
template <typename T> constexpr int unit_rows() { return 16 / (int)sizeof(T); }
template <typename T, int kHeads> constexpr int unit_tokens() {
  return 2 * unit_rows<T>() / kHeads;
}
// Tokens of one step of a CTA, (token, frequency) entries of its table.
template <typename T, int kHeads> constexpr int max_tokens() {
  return unit_tokens<T, kHeads>() == 1 ? 8 : 32;
}
template <typename T, int kHeads> constexpr int table_size() {
  return max_tokens<T, kHeads>() * kD / 2;
}

// The part of f / (2 pi) behind the point, in 2^-64 and modulo 1.  1 / (2 pi) as two doubles, off
// by 2^-110, so the part is off by less than 2^-63 + |f| 2^-107: a position of 2^31 keeps its phase
// next to any frequency up to 2^40.  Taken of |f|, whose point the double u holds exactly, and
// negated; `rest`, which passes 1 from |f| = 2^54 on, loses its whole turns as well.
__device__ __forceinline__ uint64_t turns_of(float f) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double x = fabs((double)f), u = x * kHi;
  double rest = fma(x, kHi, -u) + x * kLo;
  rest -= rint(rest);
  const uint64_t t = __double2ull_rz((u - floor(u)) * 0x1p64) + (uint64_t)__double2ll_rn(rest * 0x1p64);
  return f < 0.f ? 0ull - t : t;
}
// cos and sin of p turns: the upper 32 bits, signed, are within half a turn of 0.  `bad` is 0,
// or NaN for a frequency that is not finite.
__device__ __forceinline__ float2 cos_sin_turns(int32_t p, uint64_t turns, float bad) {
  const uint64_t x = (uint64_t)(int64_t)p * turns + 0x80000000ull;
  float s, c;
  sincospif(fmaf((float)(int32_t)(x >> 32), 0x1p-31f, bad), &s, &c);
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
  float eps;
  int n_axes, F, Hq, Hk;
  int tokens;                 // of one step of a CTA
  int splits;                 // CTAs that share a step's heads (few tokens)
};

// The raw words of 8 channels: 4 (bf16 pairs) or 8 (fp32).
template <typename T> struct Words { static constexpr int n = sizeof(T) * 2; };
__device__ __forceinline__ void load_words(const __nv_bfloat16* p, uint32_t (&w)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
}
__device__ __forceinline__ void load_words(const float* p, uint32_t (&w)[8]) {
  const uint4 u = reinterpret_cast<const uint4*>(p)[0], v = reinterpret_cast<const uint4*>(p)[1];
  w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
}
// channels 2 i and 2 i + 1
__device__ __forceinline__ float2 pair_of(const uint32_t (&w)[4], int i) {
  return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(const uint32_t (&w)[8], int i) {
  return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}

template <typename T, bool kInter, bool kNorm, int kHeads>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) norm_rope_kernel(const RopeArgs a,
                                                                           int* err) {
  constexpr int kW = Words<T>::n, kBatch = unit_rows<T>();
  constexpr bool kShared = kHeads == 2 * kBatch;
  constexpr int kRun = kShared ? kBatch : kHeads;  // rows of a half warp and token
  constexpr int kTokens = unit_tokens<T, kHeads>(), kStep = kShared ? 2 : 1;
  // (cos, sin) of (token, frequency) and the norm weights of q and k, both laid out by the
  // lane that reads them: what lanes read together is contiguous
  __shared__ __align__(16) float2 cs[2][table_size<T, kHeads>()];
  __shared__ __align__(16) float2 ws[2][kD / 2];
  struct Freq {
    uint64_t turns;
    float bad;
    int axis, place;
  };
  __shared__ Freq fr[kD / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x / a.splits, split = blockIdx.x - group * a.splits;
  // steps of a.tokens tokens, strided over the CTAs: what is read at one time lies together
  // (even shares of adjacent tokens took 137 us against 129 at 8192 tokens x 192 heads)
  const int64_t step = (int64_t)(gridDim.x / a.splits) * a.tokens;
  int64_t t0 = (int64_t)group * a.tokens;
  // half-split: lane l takes frequencies 8 l .. + 7 as four pairs; interleaved: 4 l .. + 3
  auto place = [&](int i) {
    return kInter ? (i & 3) * (a.F >> 2) + (i >> 2)
                  : 2 * (((i & 7) >> 1) * (a.F >> 3) + (i >> 3)) + (i & 1);
  };
  const int fi = tid & (kD / 2 - 1);  // this thread's frequency
  auto table = [&](int64_t t0, int buf) {
    const int nt = (int)min((int64_t)a.tokens, a.n_tokens - t0);
    if (fi >= a.F) return;
    const Freq f = fr[fi];
    const int32_t* pos = a.pos + f.axis * a.n_tokens + t0;
#pragma unroll 1
    for (int t = tid / (kD / 2); t < nt; t += kRopeThreads / (kD / 2))
      cs[buf][t * a.F + f.place] = cos_sin_turns(__ldg(pos + t), f.turns, f.bad);
  };
  if (tid < a.F) {
    const float f = __ldg(a.freq + tid);
    int ax = a.axis ? __ldg(a.axis + tid) : 0;
    if (ax < 0 || ax >= a.n_axes) {  // reported; axis 0 keeps the read in bounds
      if (err) atomicExch(err, kDevErrBadAxis);
      ax = 0;
    }
    fr[tid] = Freq{turns_of(f), f - f, ax, place(tid)};
  }
  __syncthreads();
  if (tid < kD) {  // channels 2 c, 2 c + 1 of q (first 64 threads) and k
    const float* w = tid < kD / 2 ? a.wq : a.wk;
    const int c = tid & (kD / 2 - 1);
    ws[tid / (kD / 2)][(c & 3) * 16 + (c >> 2)] =
        w ? make_float2(w[2 * c], w[2 * c + 1]) : make_float2(1.f, 1.f);
  }
  if (t0 < a.n_tokens) table(t0, 0);
  __syncthreads();
  const int hl = lane & 15, hf = lane >> 4;  // channels 8 hl .. 8 hl + 7 of every other head
  const int F8 = a.F >> 3;
  const bool rot = hl < 2 * F8, low = hl < F8;
  // half-split pairs: the lane (of the half warp) with the other channels
  const int other = kInter || !rot ? hl : (low ? hl + F8 : hl - F8);
  const int uq = (a.Hq + kHeads - 1) / kHeads, uk = (a.Hk + kHeads - 1) / kHeads;
  const int U = uq + uk;
#pragma unroll 1
  for (int buf = 0; t0 < a.n_tokens; t0 += step, buf ^= 1) {
    const int nt = (int)min((int64_t)a.tokens, a.n_tokens - t0);
#pragma unroll 1
    for (int u = warp + kRopeWarps * split; u < (nt + kTokens - 1) / kTokens * U;
         u += kRopeWarps * a.splits) {
      const int ut = u / U, ub = u - ut * U;
      const int t = kShared ? ut : kTokens * ut + hf * (kTokens / 2);
      const bool isq = ub < uq;
      const int H = isq ? a.Hq : a.Hk, h0 = (isq ? ub : ub - uq) * kHeads + (kShared ? hf : 0);
      const T* src = (isq ? static_cast<const T*>(a.q) + (t0 + t) * a.sq
                          : static_cast<const T*>(a.k) + (t0 + t) * a.sk) + h0 * kD + 8 * hl;
      T* dst = (isq ? static_cast<T*>(a.qo) + (t0 + t) * a.sqo
                    : static_cast<T*>(a.ko) + (t0 + t) * a.sko) + h0 * kD + 8 * hl;
      const int left = H - h0;
      // row b of a half warp: its token (all in the step where the half warps share one), its head
      auto row = [&](int b) {
        return (kShared || t + b / kRun < nt) && b % kRun * kStep < left;
      };
      auto at = [&](int b, int64_t sq, int64_t sk) {
        return (kRun == kBatch ? 0 : b / kRun * (isq ? sq : sk)) + b % kRun * (kStep * kD);
      };
      uint32_t x[kBatch][kW];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
#pragma unroll
        for (int i = 0; i < kW; ++i) x[b][i] = 0u;
        if (row(b)) load_words(src + at(b, a.sq, a.sk), x[b]);
      }
      // this lane's coefficients (pairs of channels) for a token's rows
      float2 A[4], B[4];
      auto coefficients = [&](int t) {
        const float2* c = cs[buf] + (kShared || t < nt ? t : 0) * a.F;
        const float2* w = ws[isq ? 0 : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 wo = w[16 * i + hl];
          if (!rot) {
            A[i] = wo;
            B[i] = make_float2(0.f, 0.f);
          } else if (kInter) {
            const float2 z = c[i * (a.F >> 2) + hl];
            A[i] = make_float2(wo.x * z.x, wo.y * z.x);
            B[i] = make_float2(-wo.y * z.y, wo.x * z.y);
          } else {
            const float2 wp = w[16 * i + other];
            const float4 z = *reinterpret_cast<const float4*>(c + 2 * (i * F8 + (low ? hl : other)));
            const float sg = low ? -1.f : 1.f;
            A[i] = make_float2(wo.x * z.x, wo.y * z.z);
            B[i] = make_float2(sg * wp.x * z.y, sg * wp.y * z.w);
          }
        }
      };
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (b % kRun == 0) coefficients(t + b / kRun);
        float r = 1.f;
        if (kNorm) {
          float2 ss = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 z = pair_of(x[b], i);
            ss = __ffma2_rn(z, z, ss);
          }
          float s = ss.x + ss.y;
#pragma unroll
          for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          r = rsqrtf(s * (1.f / kD) + a.eps);
        }
        uint32_t xp[kW];  // the other channels of this lane's pairs, as they came
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          xp[i] = x[b][i];
          if (!kInter) xp[i] = __shfl_sync(0xffffffffu, xp[i], other, 16);
          if (!rot) xp[i] = 0u;
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 p = pair_of(xp, i);
          if (kInter) p = make_float2(p.y, p.x);
          const float2 z = __fmul2_rn(
              __ffma2_rn(pair_of(x[b], i), A[i], __fmul2_rn(p, B[i])), make_float2(r, r));
          y[2 * i] = z.x;
          y[2 * i + 1] = z.y;
        }
        if (row(b)) store8(dst + at(b, a.sqo, a.sko), y);
      }
    }
    if (t0 + step < a.n_tokens) table(t0 + step, buf ^ 1);
    __syncthreads();
  }
}

int units_of_token(const RopeArgs& a, int heads) {
  return (a.Hq + heads - 1) / heads + (a.Hk + heads - 1) / heads;
}

template <typename T, int kHeads>
cudaError_t launch_rope_heads(RopeArgs a, bool inter, bool norm, int64_t most, int* err,
                              cudaStream_t s) {
  constexpr int kTokens = unit_tokens<T, kHeads>();
  const int U = units_of_token(a, kHeads);
  auto units = [&](int tokens) { return (tokens + kTokens - 1) / kTokens * U; };
  // tokens of a step: the fewest whose units fill the CTA's warps evenly, while there are
  // steps enough for every CTA (32 + 8 heads, one token a step -> this rule: 1024 tokens 8.6 ->
  // 7.6 us, 16384 tokens 106 -> 61.5)
  a.tokens = 1;
  while (a.tokens < max_tokens<T, kHeads>() &&
         (a.tokens < kTokens || units(a.tokens) % kRopeWarps != 0) &&
         a.n_tokens >= 2 * a.tokens * most)
    a.tokens *= 2;
  const int64_t steps = (a.n_tokens + a.tokens - 1) / a.tokens;
  // few tokens: their heads are spread over several CTAs (one token, 96 + 96 heads: 5.3 us in
  // one CTA, 3.9 spread)
  a.splits = 1;
  while (steps * a.splits * 2 <= most && a.splits * kRopeWarps < units(a.tokens)) a.splits *= 2;
  const int64_t groups = steps < most / a.splits ? steps : most / a.splits;
  using Fn = void (*)(const RopeArgs, int*);
  static const Fn fn[2][2] = {
      {norm_rope_kernel<T, false, false, kHeads>, norm_rope_kernel<T, false, true, kHeads>},
      {norm_rope_kernel<T, true, false, kHeads>, norm_rope_kernel<T, true, true, kHeads>}};
  fn[inter][norm]<<<(unsigned)(groups * a.splits), kRopeThreads, 0, s>>>(a, err);
  return cudaGetLastError();
}

// Heads of a token in a unit: as many as fit (every row of a warp shares one token's
// coefficients), or fewer where that leaves enough fewer rows of units empty and there are
// tokens for them.  bf16, 16 -> 8 heads: 8 + 1 heads x 16384 tokens (16 of 32 rows) 29.6 -> 18.9
// us, 16 + 2 (24 of 32) 38 -> 33, 24 + 4 (32 of 48) 48.5 -> 45, but 32 + 8 (40 of 48) 58 -> 63;
// 8 -> 2 heads: 1 + 1 x 65536 55 -> 31, 4 + 2 (6 of 16) 62 -> 48, 6 + 3 x 40000 (10 of 16) 47 -> 55.
template <typename T>
cudaError_t launch_rope_t(const RopeArgs& a, bool inter, bool norm, int* err, cudaStream_t s) {
  int sms = 152, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t most = (int64_t)sms * kRopeCtas;
  constexpr int R = unit_rows<T>();
  const int64_t all = (int64_t)units_of_token(a, 2 * R) * 2 * R,
                half = (int64_t)units_of_token(a, R) * R;
  if constexpr (R == 8) {  // (of fp32's 4 heads 2 never leave enough fewer rows empty)
    const int64_t two = (int64_t)units_of_token(a, 2) * 2;
    if (5 * two <= 2 * half && a.n_tokens >= unit_tokens<T, 2>() * most)
      return launch_rope_heads<T, 2>(a, inter, norm, most, err, s);
  }
  if (4 * half <= 3 * all && a.n_tokens >= 2 * most)
    return launch_rope_heads<T, R>(a, inter, norm, most, err, s);
  return launch_rope_heads<T, 2 * R>(a, inter, norm, most, err, s);
}

}  // namespace

cudaError_t launch_norm_rope(const void* q, const void* k, int bf16, const float* wq,
                             const float* wk, float eps, const int32_t* pos, int n_axes,
                             const int32_t* axis, const float* freq, int F, int interleaved,
                             void* qo, void* ko, int64_t n_tokens, int Hq, int Hk, int64_t sq,
                             int64_t sk, int64_t sqo, int64_t sko, int* err, cudaStream_t s) {
  const RopeArgs a{q, k, qo, ko, wq, wk, pos, axis, freq, n_tokens, sq, sk, sqo, sko, eps, n_axes,
                   F, Hq, Hk, 1, 1};
  ProfScope prof_scope("kda_qk_norm_rope", s);
  return bf16 ? launch_rope_t<__nv_bfloat16>(a, interleaved != 0, eps >= 0.f, err, s)
              : launch_rope_t<float>(a, interleaved != 0, eps >= 0.f, err, s);
}

}  // namespace kda
