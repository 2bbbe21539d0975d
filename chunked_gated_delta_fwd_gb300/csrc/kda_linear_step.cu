// kda_linear_step.cu -- new tokens of linear attention with a decay for each head, N x H
// independent states updated in place:
//     S <- e^{g_t} S + k_t v_t^T,   o_t = scale S^T q_t,   t = 0 .. T-1 (T <= 16)
//
// The state is stored transposed, S^T [dv][dk] fp32: row j is 128 contiguous floats and
// rows are independent of one another,
//     s_j <- e^{g_t} s_j + v_t[j] k_t,   o_t[j] = scale (q_t . s_j),
// so a row walks all T tokens in registers between its one load and its one store.  The
// state is stored as it is after the first n_advance tokens, the outputs of all T are
// written (the verify and the commit pass of speculative decoding in one).
//
// Bound by HBM: 2 x 64 KiB of state per head (one token, 512 x 96 states: 930 us, 7.0 TB/s;
// 5 tokens of 96 x 48 states: 92 us, 6.8 TB/s).  Eight lanes share a row (four 16-byte
// pieces a lane, each warp access four whole 128-byte segments), a lane keeps kSlots rows in
// flight, and the rows' dot products meet by a halving exchange inside the eight lanes.
// Fewer lanes a row than a warp's 32 keep the exchange short: 4 shuffles for 16 rows.  The
// tokens' vectors sit in shared memory and the products are packed pairs, which keeps the
// token walk behind the state's traffic (5 tokens: 114 us with v read from global memory
// row by row, 98 us with single products).
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kLsThreads = 128;
constexpr int kSlots = 4;                       // rows of a lane in flight
constexpr int kPassRows = 4 * (kLsThreads / 32) * kSlots;  // 64 rows of a CTA's pass
constexpr int kLsMaxT = 16;

template <typename T, bool kMulti>
__global__ void __launch_bounds__(kLsThreads) linear_step_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ g, int g_head, float scale, float* __restrict__ S,
    T* __restrict__ o, const int32_t* __restrict__ n_advance, int H, int rep, int Tn) {
  constexpr int kT = kMulti ? kLsMaxT : 1;
  __shared__ __align__(16) float tq[kT][kD], tk[kT][kD], tv[kT][kD];
  __shared__ float ta[kT];
  const int64_t unit = blockIdx.x;  // n * H + h
  const int n = (int)(unit / H), h = (int)(unit - (int64_t)n * H);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = h / rep, Hk = H / rep;
  const int nT = kMulti ? Tn : 1;
  int adv = nT;
  if (kMulti && n_advance) {
    adv = __ldg(n_advance + n);
    adv = adv < 0 ? 0 : (adv > nT ? nT : adv);
  }
  const int sub = lane & 7, grp = lane >> 3;  // piece of the row, row of the warp's four
  const int row0 = blockIdx.y * (kD / gridDim.y);
  float4* Su = reinterpret_cast<float4*>(S + unit * kD * kD);
  auto row_of = [&](int pass, int i) { return row0 + pass * kPassRows + 16 * warp + 4 * i + grp; };
  float4 s[kSlots][4];
  auto load_pass = [&](int pass) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) s[i][m] = __ldcs(Su + row_of(pass, i) * (kD / 4) + 8 * m + sub);
  };
  load_pass(0);  // in flight while the tokens' vectors are laid out
  for (int e = tid; e < nT * (kD / 4); e += kLsThreads) {
    const int t = e / (kD / 4), c = 4 * (e % (kD / 4));
    const int64_t row = ((int64_t)n * nT + t) * Hk + hk;
    float x[4];
    load4(q + row * kD + c, x);
    *reinterpret_cast<float4*>(&tq[t][c]) =
        make_float4(scale * x[0], scale * x[1], scale * x[2], scale * x[3]);
    load4(k + row * kD + c, x);
    *reinterpret_cast<float4*>(&tk[t][c]) = make_float4(x[0], x[1], x[2], x[3]);
    load4(v + (((int64_t)n * nT + t) * H + h) * kD + c, x);
    *reinterpret_cast<float4*>(&tv[t][c]) = make_float4(x[0], x[1], x[2], x[3]);
  }
  if (tid < nT) ta[tid] = expf(__ldg(g + (g_head ? (int64_t)h : ((int64_t)n * nT + tid) * H + h)));
  __syncthreads();
  const int passes = kD / gridDim.y / kPassRows;
  for (int pass = 0; pass < passes; ++pass) {
    if (pass > 0) load_pass(pass);
#pragma unroll 1
    for (int t = 0; t < nT; ++t) {
      const int64_t vrow = (((int64_t)n * nT + t) * H + h) * kD;
      const float2 aa = make_float2(ta[t], ta[t]);
      float vj[kSlots], d[kSlots];
      float2 d2[kSlots];  // even and odd channels apart: packed products
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        vj[i] = tv[t][row_of(pass, i)];
        d2[i] = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float4 kk = *reinterpret_cast<const float4*>(&tk[t][32 * m + 4 * sub]);
        const float4 qq = *reinterpret_cast<const float4*>(&tq[t][32 * m + 4 * sub]);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          float4& x = s[i][m];
          const float2 vv = make_float2(vj[i], vj[i]);
          const float2 lo =
              __ffma2_rn(vv, make_float2(kk.x, kk.y), __fmul2_rn(aa, make_float2(x.x, x.y)));
          const float2 hi =
              __ffma2_rn(vv, make_float2(kk.z, kk.w), __fmul2_rn(aa, make_float2(x.z, x.w)));
          d2[i] = __ffma2_rn(make_float2(qq.x, qq.y), lo,
                             __ffma2_rn(make_float2(qq.z, qq.w), hi, d2[i]));
          x = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
#pragma unroll
      for (int i = 0; i < kSlots; ++i) d[i] = d2[i].x + d2[i].y;
      if (t + 1 == adv) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) __stcs(Su + row_of(pass, i) * (kD / 4) + 8 * m + sub, s[i][m]);
      }
      if (o) {  // halving exchange over the eight lanes: lane sub ends with slot sub >> 1
        const bool u4 = (sub & 4) != 0, u2 = (sub & 2) != 0;
        float e0 = (u4 ? d[2] : d[0]) + __shfl_xor_sync(0xffffffffu, u4 ? d[0] : d[2], 4);
        float e1 = (u4 ? d[3] : d[1]) + __shfl_xor_sync(0xffffffffu, u4 ? d[1] : d[3], 4);
        float y = (u2 ? e1 : e0) + __shfl_xor_sync(0xffffffffu, u2 ? e0 : e1, 2);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        if ((sub & 1) == 0) o[vrow + row_of(pass, sub >> 1)] = from_f32<T>(y);
      }
    }
  }
}

template <typename T>
void launch_step_t(const void* q, const void* k, const void* v, const float* g, int g_head,
                   float scale, float* S, void* o, const int32_t* n_advance, int N, int Tn, int H,
                   int Hk, bool multi, cudaStream_t s) {
  const int64_t units = (int64_t)N * H;
  int sms = 152, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // at most one state an SM: two CTAs share its rows, so that the latency is one pass's
  // (8, 76, 152 states, one CTA -> two: one token 3.5 -> 2.7, 3.5 -> 2.7, 3.8 -> 3.7 us,
  // 16 tokens 10.3 -> 6.4, 10.4 -> 6.5, 10.6 -> 8.7); beyond, the second CTA only repeats the
  // tokens' vectors (2 tokens, 384 states: 7.4 -> 8.0 us)
  const dim3 grid((unsigned)units, units <= sms ? 2u : 1u);
  const auto fn = multi ? linear_step_kernel<T, true> : linear_step_kernel<T, false>;
  fn<<<grid, kLsThreads, 0, s>>>(static_cast<const T*>(q), static_cast<const T*>(k),
                                 static_cast<const T*>(v), g, g_head, scale, S,
                                 static_cast<T*>(o), n_advance, H, H / Hk, Tn);
}

}  // namespace

cudaError_t launch_linear_step(const void* q, const void* k, const void* v, int bf16,
                               const float* g, int g_head, float scale, float* S, void* o,
                               const int32_t* n_advance, int N, int Tn, int H, int Hk, bool multi,
                               cudaStream_t s) {
  ProfScope prof_scope(multi ? "kda_linear_multi_step" : "kda_linear_step", s);
  if (bf16)
    launch_step_t<__nv_bfloat16>(q, k, v, g, g_head, scale, S, o, n_advance, N, Tn, H, Hk, multi, s);
  else
    launch_step_t<float>(q, k, v, g, g_head, scale, S, o, n_advance, N, Tn, H, Hk, multi, s);
  return cudaGetLastError();
}

}  // namespace kda
