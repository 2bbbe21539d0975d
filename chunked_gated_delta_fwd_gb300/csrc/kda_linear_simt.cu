// kda_linear_simt.cu -- the prompt pass of linear attention with a decay for each head,
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// on fp32 CUDA cores: the path of fp32 inputs, and a cross-check of the tensor-core path
// for bf16 ones.  In chunks of 64 tokens, G the running sum of g inside a chunk:
//     local = sum_j e^{G_C - G_j} k_j v_j^T              (every chunk on its own)
//     S_in  = running state over the chunks' locals       (elementwise scan)
//     O_i   = scale (e^{G_i} S_in^T q_i + sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j)
// Three launches after the plan.  Only the scan walks a sequence in order, and it does
// nothing but add: products over the whole prompt run at once, also with one head.
//
// Exponents are differences of running sums.  A gate may take g to -inf, so g is held at
// -200 at least (e^-200 is 0 in fp32) and the sums as an exact pair of floats (a multiple
// of 2^-8 and the rest): differences keep fp32 accuracy next to a g of -200.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int C = kChunk;   // 64
constexpr int D = kD;       // 128
constexpr int LD = D + 4;   // padded row of a shared tile
constexpr float kMinG = -200.f;

// NaN stays NaN
__device__ __forceinline__ float clamp_g(float g) { return g < kMinG ? kMinG : g; }

struct Sums {       // running sums of a chunk's g: hi + lo, hi a multiple of 2^-8
  float hi[C], lo[C];
};

// Threads 0..63 (two whole warps) fill `sm` from the chunk's g; rows past `len` repeat
// the last sum.  Ends with a barrier over the CTA.
__device__ __forceinline__ void chunk_sums(Sums& sm, double* half, const float* __restrict__ g,
                                           int g_head, int64_t t0, int len, int H, int h) {
  const int t = threadIdx.x;
  double x = 0.0;
  if (t < C) {
    if (t < len) x = (double)clamp_g(__ldg(g + (g_head ? (int64_t)h : (t0 + t) * H + h)));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if ((t & 31) >= o) x += y;
    }
    if (t == 31) *half = x;
  }
  __syncthreads();
  if (t < C) {
    if (t >= 32) x += *half;
    const float hi = (float)(rint(x * 256.0) * (1.0 / 256.0));
    sm.hi[t] = hi;
    sm.lo[t] = (float)(x - (double)hi);
  }
  __syncthreads();
}
__device__ __forceinline__ float decay(const Sums& s, int i, int j) {
  return expf((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j]));
}
__device__ __forceinline__ float decay_from_start(const Sums& s, int i) {
  return expf(s.hi[i] + s.lo[i]);
}

// rows t0 .. t0 + len - 1 of one head, columns c0 .. c0 + W - 1, zero rows up to `rows`
template <typename T, int W, int LDW, int kThreads>
__device__ __forceinline__ void load_tile(float (*dst)[LDW], const T* __restrict__ x, int64_t t0,
                                          int rows, int len, int heads, int head, int c0) {
  for (int e = threadIdx.x; e < rows * (W / 4); e += kThreads) {
    const int r = e / (W / 4), c = 4 * (e % (W / 4));
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < len) load4(x + ((t0 + r) * heads + head) * D + c0 + c, y);
    *reinterpret_cast<float4*>(&dst[r][c]) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

// ------------------------------------------------------------------ local states
// One CTA per (chunk, head, 64 x 64 quarter): quarters let a short prompt with few heads
// occupy four times the SMs; thread = 8 value rows x 4 key columns.
constexpr int kLocThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kLocThreads) lin_local_kernel(
    const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ g, int g_head,
    Plan plan, int H, int Hk, float* __restrict__ local, float* __restrict__ gam) {
  constexpr int LQ = 64 + 4;
  __shared__ __align__(16) float Ks[C][LQ], Vs[C][LQ];
  __shared__ Sums sums;
  __shared__ double half;
  const int chunk = blockIdx.x, h = blockIdx.y, v0 = 64 * (blockIdx.z >> 1),
            k0 = 64 * (blockIdx.z & 1), tid = threadIdx.x;
  if (chunk >= __ldg(plan.chunk_off + plan.n_seqs)) return;
  const int2 e = plan.tab[chunk];
  const int64_t t0 = e.x;
  const int len = e.y, hk = h / (H / Hk);
  load_tile<T, 64, LQ, kLocThreads>(Ks, k, t0, C, len, Hk, hk, k0);
  load_tile<T, 64, LQ, kLocThreads>(Vs, v, t0, C, len, H, h, v0);
  chunk_sums(sums, &half, g, g_head, t0, len, H, h);
  for (int x = tid; x < C * 16; x += kLocThreads) {
    const int r = x >> 4, c = 4 * (x & 15);
    const float w = decay(sums, C - 1, r);
    float4& y = *reinterpret_cast<float4*>(&Ks[r][c]);
    y = make_float4(w * y.x, w * y.y, w * y.z, w * y.w);
  }
  __syncthreads();
  const int vr = 8 * (tid >> 4), kc = 4 * (tid & 15);
  float2 acc[8][2] = {};
#pragma unroll 4
  for (int j = 0; j < C; ++j) {
    const float4 kk = *reinterpret_cast<const float4*>(&Ks[j][kc]);
    const float4 va = *reinterpret_cast<const float4*>(&Vs[j][vr]);
    const float4 vb = *reinterpret_cast<const float4*>(&Vs[j][vr + 4]);
    const float vv[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = make_float2(vv[i], vv[i]);
      acc[i][0] = __ffma2_rn(x, make_float2(kk.x, kk.y), acc[i][0]);
      acc[i][1] = __ffma2_rn(x, make_float2(kk.z, kk.w), acc[i][1]);
    }
  }
  const int64_t unit = (int64_t)chunk * H + h;
  float* out = local + unit * D * D;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(out + (v0 + vr + i) * D + k0 + kc) =
        make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
  if (blockIdx.z == 0 && tid == 0) gam[unit] = decay_from_start(sums, C - 1);
}

// ----------------------------------------------------------------------- the scan
// local[c] becomes the state entering chunk c; one float4 of the state a thread, the next
// chunks' locals in flight while one is added.
constexpr int kScanThreads = 256, kScanAhead = 4;

__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(
    const float* __restrict__ h0, Plan plan, int H, float* __restrict__ local,
    const float* __restrict__ gam, float* __restrict__ hT) {
  const int64_t unit = blockIdx.x;  // n * H + h
  const int n = (int)(unit / H), h = (int)(unit - (int64_t)n * H);
  const int64_t e = 4 * ((int64_t)blockIdx.y * kScanThreads + threadIdx.x);
  const int c0 = __ldg(plan.chunk_off + n), c1 = __ldg(plan.chunk_off + n + 1);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h0) s = *reinterpret_cast<const float4*>(h0 + unit * D * D + e);
  auto at = [&](int c) {
    return reinterpret_cast<float4*>(local + ((int64_t)c * H + h) * D * D + e);
  };
  for (int c = c0; c < c1; c += kScanAhead) {
    float4 x[kScanAhead];
    float a[kScanAhead];
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (c + i < c1) {
        x[i] = *at(c + i);
        a[i] = __ldg(gam + (int64_t)(c + i) * H + h);
      }
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (c + i < c1) {
        *at(c + i) = s;
        s = make_float4(fmaf(a[i], s.x, x[i].x), fmaf(a[i], s.y, x[i].y), fmaf(a[i], s.z, x[i].z),
                        fmaf(a[i], s.w, x[i].w));
      }
  }
  if (hT) *reinterpret_cast<float4*>(hT + unit * D * D + e) = s;
}

// --------------------------------------------------------------------- the outputs
// One CTA per (chunk, head, 32 rows of the chunk): scores of its rows (32 x 64 over 128
// channels), then both products of the output, 64 value columns at a time.
constexpr int kOutThreads = 256, kOutRows = 32;

struct OutSmem {
  float Q[kOutRows][LD];
  float X[C][LD];              // k, then v, then (as [64][LD]) halves of the state
  float P[kOutRows][C + 4];
  Sums sums;
  double half;
};

template <typename T>
__global__ void __launch_bounds__(kOutThreads) lin_out_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ g, int g_head, float scale, Plan plan, int H, int Hk,
    const float* __restrict__ states, T* __restrict__ o) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  OutSmem& sm = *reinterpret_cast<OutSmem*>(smem_raw);
  const int chunk = blockIdx.x, h = blockIdx.y, r0 = kOutRows * blockIdx.z, tid = threadIdx.x;
  if (chunk >= __ldg(plan.chunk_off + plan.n_seqs)) return;
  const int2 e = plan.tab[chunk];
  const int64_t t0 = e.x;
  const int len = e.y, hk = h / (H / Hk);
  if (r0 >= len) return;
  const int cols = r0 + kOutRows;  // keys that the CTA's rows may see
  load_tile<T, D, LD, kOutThreads>(sm.Q, q, t0 + r0, kOutRows, len - r0, Hk, hk, 0);
  load_tile<T, D, LD, kOutThreads>(sm.X, k, t0, cols, len, Hk, hk, 0);
  chunk_sums(sm.sums, &sm.half, g, g_head, t0, len, H, h);
  const int ty = tid >> 4, tx = tid & 15;  // 16 x 16 threads: rows ty, ty + 16; columns tx + 16 c
  {
    float acc[2][4] = {};
    const int nc = cols / 16;  // 2 or 4 column blocks
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qa[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) qa[i] = *reinterpret_cast<const float4*>(&sm.Q[ty + 16 * i][c]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b >= nc) break;
        const float4 kk = *reinterpret_cast<const float4*>(&sm.X[tx + 16 * b][c]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][b] = fmaf(qa[i].x, kk.x,
                           fmaf(qa[i].y, kk.y, fmaf(qa[i].z, kk.z, fmaf(qa[i].w, kk.w, acc[i][b]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int r = ty + 16 * i, j = tx + 16 * b;
        if (b < nc) sm.P[r][j] = j <= r0 + r ? acc[i][b] * decay(sm.sums, r0 + r, j) : 0.f;
      }
  }
  __syncthreads();
  // O = e^G Q S: 64 value rows of S^T at a time, thread = 2 rows x 4 value columns of each half
  float out[2][2][4] = {};  // [half][row][column]
  const float* S = states + ((int64_t)chunk * H + h) * D * D;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    for (int x = tid; x < 64 * (D / 4); x += kOutThreads) {
      const int r = x / (D / 4), c = 4 * (x % (D / 4));
      *reinterpret_cast<float4*>(&sm.X[r][c]) =
          *reinterpret_cast<const float4*>(S + (64 * hf + r) * D + c);
    }
    __syncthreads();
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qa[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) qa[i] = *reinterpret_cast<const float4*>(&sm.Q[ty + 16 * i][c]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float4 ss = *reinterpret_cast<const float4*>(&sm.X[tx + 16 * b][c]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          out[hf][i][b] =
              fmaf(qa[i].x, ss.x,
                   fmaf(qa[i].y, ss.y, fmaf(qa[i].z, ss.z, fmaf(qa[i].w, ss.w, out[hf][i][b]))));
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float w = decay_from_start(sm.sums, r0 + ty + 16 * i);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      out[0][i][b] *= w;
      out[1][i][b] *= w;
    }
  }
  // O += P V
  load_tile<T, D, LD, kOutThreads>(sm.X, v, t0, cols, len, H, h, 0);
  __syncthreads();
#pragma unroll 4
  for (int j = 0; j < cols; ++j) {
    const float p0 = sm.P[ty][j], p1 = sm.P[ty + 16][j];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float x = sm.X[j][64 * hf + tx + 16 * b];
        out[hf][0][b] = fmaf(p0, x, out[hf][0][b]);
        out[hf][1][b] = fmaf(p1, x, out[hf][1][b]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + ty + 16 * i;
    if (r < len) {
      T* orow = o + ((t0 + r) * H + h) * D;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          orow[64 * hf + tx + 16 * b] = from_f32<T>(scale * out[hf][i][b]);
    }
  }
}

template <typename T>
cudaError_t launch_t(const void* q, const void* k, const void* v, const float* g, int g_head,
                     float scale, const float* h0, void* o, float* hT, int64_t n_tokens,
                     int n_seqs, int H, int Hk, void* ws, cudaStream_t s) {
  const Plan plan = plan_in(ws, n_tokens, n_seqs);
  const int64_t chunks = chunks_upper_bound(n_tokens, n_seqs);
  float* local = reinterpret_cast<float*>(static_cast<char*>(ws) + plan_bytes(n_tokens, n_seqs));
  float* gam = local + (size_t)chunks * H * D * D;
  cudaError_t e;
  if (n_tokens > 0) {
    ProfScope prof_scope("kda_linear_local", s);
    lin_local_kernel<T><<<dim3((unsigned)chunks, (unsigned)H, 4), kLocThreads, 0, s>>>(
        static_cast<const T*>(k), static_cast<const T*>(v), g, g_head, plan, H, Hk, local, gam);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  {
    ProfScope prof_scope("kda_linear_scan", s);
    lin_scan_kernel<<<dim3((unsigned)((int64_t)n_seqs * H), D * D / 4 / kScanThreads),
                      kScanThreads, 0, s>>>(h0, plan, H, local, gam, hT);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (n_tokens == 0) return cudaSuccess;
  e = cudaFuncSetAttribute(lin_out_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)sizeof(OutSmem));
  if (e != cudaSuccess) return e;
  ProfScope prof_scope("kda_linear_out", s);
  lin_out_kernel<T><<<dim3((unsigned)chunks, (unsigned)H, C / kOutRows), kOutThreads,
                      sizeof(OutSmem), s>>>(static_cast<const T*>(q), static_cast<const T*>(k),
                                            static_cast<const T*>(v), g, g_head, scale, plan, H,
                                            Hk, local, static_cast<T*>(o));
  return cudaGetLastError();
}

}  // namespace

size_t linear_simt_workspace_bytes(int64_t n_tokens, int n_seqs, int H) {
  return (size_t)chunks_upper_bound(n_tokens, n_seqs) * H * (D * D + 1) * sizeof(float);
}

cudaError_t launch_linear_simt(const void* q, const void* k, const void* v, int bf16,
                               const float* g, int g_head, float scale, const float* h0, void* o,
                               float* hT, int64_t n_tokens, int n_seqs, int H, int Hk, void* ws,
                               cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(q, k, v, g, g_head, scale, h0, o, hT, n_tokens, n_seqs, H,
                                        Hk, ws, s)
              : launch_t<float>(q, k, v, g, g_head, scale, h0, o, hT, n_tokens, n_seqs, H, Hk, ws,
                                s);
}

}  // namespace kda
