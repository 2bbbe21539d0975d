// kda_linear_simt.cu -- the prompt pass of linear attention with a decay for each head,
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// on fp32 CUDA cores: the path of fp32 inputs, and a cross-check of the tensor-core path
// for bf16 ones.  In chunks of 64 tokens, G the running sum of g inside a chunk:
//     local = sum_j e^{G_C - G_j} k_j v_j^T              (every chunk on its own)
//     S_in  = running state over the chunks' locals       (elementwise scan)
//     O_i   = scale (e^{G_i} S_in^T q_i + sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j)
// Three launches after the plan, each begun while the one before ends.  Only the scan walks a
// sequence in order, and it does nothing but add: products over the whole prompt run at once, also
// with one head.  Measured:
// 2102 tokens in five sequences, 16 heads: 104 us (plan 4, local 31, scan 19, outputs 56 one by
// one), 32 TFLOP/s; 64 tokens of one head 22 us, four launches' latency.
//
// Exponents are differences of running sums.  A gate may take g to -inf, so g is held at
// -200 at least (e^-200 is 0 in fp32) and the sums as an exact pair of floats (a multiple
// of 2^-8 and the rest): differences keep fp32 accuracy next to a g of -200.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int C = kChunk;   // 64
constexpr int D = kD;       // 128
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

// 16-byte chunk c4 of row r of a shared tile whose rows are W floats: chunks are permuted by
// r / 4, so that lanes that read the same chunk of rows 4 apart do not meet in a bank.
// kShift 0 permutes by r for lanes that read adjacent rows.
template <int W, int kShift = 2>
__device__ __forceinline__ float4& tile_at(float* tile, int r, int c4) {
  return reinterpret_cast<float4*>(tile + r * W)[c4 ^ ((r >> kShift) & 7)];
}

// Rows t0 .. t0 + len - 1 of one head, columns c0 .. c0 + W - 1, into a shared tile of R
// rows (zeros past len).  Every load is in flight before the first store.
template <typename T, int R, int W, int kThreads, int kShift = 2>
__device__ __forceinline__ void load_tile(float* dst, const T* __restrict__ x, int64_t t0, int len,
                                          int heads, int head, int c0) {
  constexpr int n = R * (W / 4) / kThreads;
  static_assert(n * kThreads == R * (W / 4), "whole loads a thread");
  float y[n][4];
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / (W / 4), c = 4 * (e % (W / 4));
    y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
    if (r < len) load4(x + ((t0 + r) * heads + head) * D + c0 + c, y[i]);
  }
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const int e = threadIdx.x + i * kThreads;
    tile_at<W, kShift>(dst, e / (W / 4), e % (W / 4)) =
        make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
  }
}

// The same for fp32 without a stop in registers: the copies are on their way when this returns
// (bf16 is converted, and is in place).
template <int R, int kThreads, int kShift = 2>
__device__ __forceinline__ void start_tile(float* dst, const float* x, int64_t t0, int len,
                                           int heads, int head) {
#pragma unroll
  for (int i = 0; i < R * (D / 4) / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / (D / 4), c4 = e % (D / 4);
    const float* src = x + ((t0 + (r < len ? r : 0)) * heads + head) * D + 4 * c4;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(&tile_at<D, kShift>(dst, r, c4));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src),
                 "r"(r < len ? 16 : 0)  // no bytes read: zeros
                 : "memory");
  }
}
template <int R, int kThreads, int kShift = 2>
__device__ __forceinline__ void start_tile(float* dst, const __nv_bfloat16* __restrict__ x,
                                           int64_t t0, int len, int heads, int head) {
  load_tile<__nv_bfloat16, R, D, kThreads, kShift>(dst, x, t0, len, heads, head, 0);
}
__device__ __forceinline__ void commit_tiles() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void wait_tiles() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// ------------------------------------------------------------------ local states
// One CTA per (chunk, head, 64 value rows); thread = 8 value rows x 4 key columns of each
// 64: 4 shared-memory reads of 16 bytes for 32 packed products.  Keys go to shared memory by
// themselves while the decays are formed, values by way of the registers where they are weighted
// (1024 chunks x heads, the whole pass: 179 us with a second trip for the weights, 174).
constexpr int kLocThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kLocThreads) lin_local_kernel(
    const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ g, int g_head,
    Plan plan, int H, int Hk, float* __restrict__ local, float* __restrict__ gam) {
  constexpr int G = D / 64;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* Ks = reinterpret_cast<float*>(smem_raw);  // [C][D]
  float* Vs = Ks + C * D;                         // [C][64]
  __shared__ Sums sums;
  __shared__ double half;
  const int chunk = blockIdx.x, h = blockIdx.y, v0 = 64 * blockIdx.z, tid = threadIdx.x;
  wait_previous();
  if (chunk >= plan.chunk_off[plan.n_seqs]) return;
  const int2 e = plan.tab[chunk];
  const int64_t t0 = e.x;
  const int len = e.y, hk = h / (H / Hk);
  start_tile<C, kLocThreads>(Ks, k, t0, len, Hk, hk);
  commit_tiles();
  constexpr int n = C * 16 / kLocThreads;
  float y[n][4];
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const int r = (tid >> 4) + i * (kLocThreads / 16);
    y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
    if (r < len) load4(v + ((t0 + r) * H + h) * D + v0 + 4 * (tid & 15), y[i]);
  }
  chunk_sums(sums, &half, g, g_head, t0, len, H, h);
#pragma unroll
  for (int i = 0; i < n; ++i) {  // v_j times its decay to the chunk's end
    const int r = (tid >> 4) + i * (kLocThreads / 16);
    const float w = decay(sums, C - 1, r);
    tile_at<64>(Vs, r, tid & 15) = make_float4(w * y[i][0], w * y[i][1], w * y[i][2], w * y[i][3]);
  }
  wait_tiles<0>();
  __syncthreads();
  const int vr = 8 * (tid >> 4), tx = tid & 15;
  float2 acc[8][G][2] = {};
#pragma unroll 4
  for (int j = 0; j < C; ++j) {
    const float4 va = tile_at<64>(Vs, j, vr >> 2);
    const float4 vb = tile_at<64>(Vs, j, (vr >> 2) + 1);
    const float vv[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int b = 0; b < G; ++b) {
      const float4 kk = tile_at<D>(Ks, j, 16 * b + tx);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = make_float2(vv[i], vv[i]);
        acc[i][b][0] = __ffma2_rn(x, make_float2(kk.x, kk.y), acc[i][b][0]);
        acc[i][b][1] = __ffma2_rn(x, make_float2(kk.z, kk.w), acc[i][b][1]);
      }
    }
  }
  release_next();
  const int64_t unit = (int64_t)chunk * H + h;
  float* out = local + unit * D * D;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int b = 0; b < G; ++b)
      *reinterpret_cast<float4*>(out + (v0 + vr + i) * D + 64 * b + 4 * tx) =
          make_float4(acc[i][b][0].x, acc[i][b][0].y, acc[i][b][1].x, acc[i][b][1].y);
  if (blockIdx.z == 0 && tid == 0) gam[unit] = decay_from_start(sums, C - 1);
}

template <typename T>
cudaError_t launch_local(const void* k, const void* v, const float* g, int g_head,
                         const Plan& plan, int64_t chunks, int H, int Hk, float* local,
                         float* gam, cudaStream_t s) {
  constexpr int smem = C * (D + 64) * (int)sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(lin_local_kernel<T>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof_scope("kda_linear_local", s);
  return launch_chained(lin_local_kernel<T>, dim3((unsigned)chunks, (unsigned)H, D / 64),
                        kLocThreads, smem, s, static_cast<const T*>(k), static_cast<const T*>(v),
                        g, g_head, plan, H, Hk, local, gam);
}

// ----------------------------------------------------------------------- the scan
// local[c] becomes the state entering chunk c; one float4 of the state a thread, eight
// chunks' locals in flight, the next eight on their way while eight are added.
constexpr int kScanThreads = 256, kScanAhead = 8;

__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(
    const float* h0, Plan plan, int H, float* local, const float* gam, float* hT) {
  const int64_t unit = blockIdx.x;  // n * H + h
  const int n = (int)(unit / H), h = (int)(unit - (int64_t)n * H);
  const int64_t e = 4 * ((int64_t)blockIdx.y * kScanThreads + threadIdx.x);
  wait_previous();
  const int c0 = plan.chunk_off[n], c1 = plan.chunk_off[n + 1];
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h0) s = *reinterpret_cast<const float4*>(h0 + unit * D * D + e);
  auto at = [&](int c) {
    return reinterpret_cast<float4*>(local + ((int64_t)c * H + h) * D * D + e);
  };
  float4 x[2][kScanAhead];
  float a[2][kScanAhead];
  auto fetch = [&](int b, int c) {
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (c + i < c1) {
        x[b][i] = *at(c + i);
        a[b][i] = gam[(int64_t)(c + i) * H + h];
      }
  };
  fetch(0, c0);
  for (int c = c0; c < c1; c += 2 * kScanAhead) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int cb = c + b * kScanAhead;
      fetch(b ^ 1, cb + kScanAhead);
#pragma unroll
      for (int i = 0; i < kScanAhead; ++i)
        if (cb + i < c1) {
          *at(cb + i) = s;
          s = make_float4(fmaf(a[b][i], s.x, x[b][i].x), fmaf(a[b][i], s.y, x[b][i].y),
                          fmaf(a[b][i], s.z, x[b][i].z), fmaf(a[b][i], s.w, x[b][i].w));
        }
    }
  }
  release_next();
  if (hT) *reinterpret_cast<float4*>(hT + unit * D * D + e) = s;
}

// --------------------------------------------------------------------- the outputs
// One CTA per (chunk, head, kR rows of the chunk): scores of its rows over 128 channels, then
// both products of the output.  A thread owns kR / 8 rows and four adjacent columns of each
// 64 (keys, then value columns): 8 x 16 threads.  Products over channels run on pairs of
// channels, products over keys on pairs of columns (packed fp32).  The next tile is copied
// while one is multiplied.  1024 chunks x heads, the whole pass: 205 us with copies and
// products in turn and 16 x 16 threads of four rows, 199 with copies ahead, 195 with eight rows
// a thread (12 reads of 16 bytes a lane feed 64 packed products), 178 with the products above
// the diagonal left out by blocks of 8 rows x 16 keys.  kR = 64 reads each operand from shared
// memory least often; kR = 16 gives the shortest prompts four times the CTAs.
constexpr int kOutThreads = 128;

template <int kR>
struct OutSmem {
  float Q[kR * D];
  float X[2][C * D];  // k and half a state's rows, then the other half and v
  float P[kR * C];
  Sums sums;
  double half;
};

// acc[i][b] = row ty + 8 i of Q . row 4 tx + b of X, over 128 channels.  For scores it is row
// tx + 16 b: all lanes then skip the keys that none of their rows i may see (12 of the 32
// products of a whole chunk).
template <int kR, bool kScores>
__device__ __forceinline__ void dot_tile(float (&acc)[kR / 8][4], float* Q, float* X, int ty,
                                         int tx) {
  constexpr int R = kR / 8;
  float2 a2[R][4] = {};
#pragma unroll 2
  for (int c = 0; c < D / 4; ++c) {
    float4 qa[R];
#pragma unroll
    for (int i = 0; i < R; ++i) qa[i] = tile_at<D>(Q, ty + 8 * i, c);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 x = kScores ? tile_at<D, 0>(X, tx + 16 * b, c) : tile_at<D>(X, 4 * tx + b, c);
#pragma unroll
      for (int i = kScores && kR == C ? 2 * b : 0; i < R; ++i)
        a2[i][b] = __ffma2_rn(make_float2(qa[i].x, qa[i].y), make_float2(x.x, x.y),
                              __ffma2_rn(make_float2(qa[i].z, qa[i].w), make_float2(x.z, x.w),
                                         a2[i][b]));
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[i][b] = a2[i][b].x + a2[i][b].y;
}

template <typename T, int kR>
__global__ void __launch_bounds__(kOutThreads, 2) lin_out_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ g, int g_head, float scale, Plan plan, int H, int Hk,
    const float* states, T* __restrict__ o) {
  constexpr int R = kR / 8;  // rows of a thread: ty + 8 i
  extern __shared__ __align__(16) unsigned char smem_raw[];
  OutSmem<kR>& sm = *reinterpret_cast<OutSmem<kR>*>(smem_raw);
  const int chunk = blockIdx.x, h = blockIdx.y, r0 = kR * blockIdx.z, tid = threadIdx.x;
  wait_previous();
  if (chunk >= plan.chunk_off[plan.n_seqs]) return;
  const int2 e = plan.tab[chunk];
  const int64_t t0 = e.x;
  const int len = e.y, hk = h / (H / Hk);
  if (r0 >= len) return;
  const float* S = states + ((int64_t)chunk * H + h) * D * D;
  start_tile<kR, kOutThreads>(sm.Q, q, t0 + r0, len - r0, Hk, hk);
  start_tile<C, kOutThreads, 0>(sm.X[0], k, t0, len, Hk, hk);
  commit_tiles();
  start_tile<C, kOutThreads>(sm.X[1], S, 0, C, 1, 0);
  commit_tiles();
  chunk_sums(sm.sums, &sm.half, g, g_head, t0, len, H, h);
  const int ty = tid >> 4, tx = tid & 15;
  const int cols = min(C, r0 + kR);  // keys that these rows may see
  wait_tiles<1>();
  __syncthreads();
  {
    float acc[R][4];
    dot_tile<kR, true>(acc, sm.Q, sm.X[0], ty, tx);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (kR == C && i < 2 * b) continue;  // not read either
        const int r = ty + 8 * i, j = tx + 16 * b;
        sm.P[r * C + j] = j <= r0 + r ? acc[i][b] * decay(sm.sums, r0 + r, j) : 0.f;
      }
  }
  // O = e^G Q S, 64 value rows of S^T at a time
  float2 out[2][R][2];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    wait_tiles<0>();
    __syncthreads();  // a tile has landed, the other's last reads are done
    if (hf == 0)
      start_tile<C, kOutThreads>(sm.X[0], S + C * D, 0, C, 1, 0);
    else
      start_tile<C, kOutThreads>(sm.X[1], v, t0, len, H, h);
    commit_tiles();
    float acc[R][4];
    dot_tile<kR, false>(acc, sm.Q, sm.X[hf ^ 1], ty, tx);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float w = decay_from_start(sm.sums, r0 + ty + 8 * i);
      out[hf][i][0] = make_float2(w * acc[i][0], w * acc[i][1]);
      out[hf][i][1] = make_float2(w * acc[i][2], w * acc[i][3]);
    }
  }
  // O += P V over the keys that these rows may see, 16 at a time
  wait_tiles<0>();
  __syncthreads();
#pragma unroll
  for (int m = 0; m < (kR == C ? C / 16 : 1); ++m) {
    const int first = 2 * m, end = kR == C ? 16 * (m + 1) : cols;  // rows i < first see none
#pragma unroll 2
    for (int j = 16 * m; j < end; j += 4) {
      float4 p[R];
#pragma unroll
      for (int i = first; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(&sm.P[(ty + 8 * i) * C + j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float4 x = tile_at<D>(sm.X[1], j + jj, 16 * hf + tx);
#pragma unroll
          for (int i = first; i < R; ++i) {
            const float pj = jj == 0 ? p[i].x : (jj == 1 ? p[i].y : (jj == 2 ? p[i].z : p[i].w));
            out[hf][i][0] = __ffma2_rn(make_float2(pj, pj), make_float2(x.x, x.y), out[hf][i][0]);
            out[hf][i][1] = __ffma2_rn(make_float2(pj, pj), make_float2(x.z, x.w), out[hf][i][1]);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + ty + 8 * i;
    if (r < len) {
      T* orow = o + ((t0 + r) * H + h) * D + 4 * tx;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float y[4] = {scale * out[hf][i][0].x, scale * out[hf][i][0].y,
                            scale * out[hf][i][1].x, scale * out[hf][i][1].y};
        store4(orow + 64 * hf, y);
      }
    }
  }
}

template <typename T, int kR>
cudaError_t launch_out(const void* q, const void* k, const void* v, const float* g, int g_head,
                       float scale, const Plan& plan, int64_t chunks, int H, int Hk,
                       const float* states, void* o, cudaStream_t s) {
  const int smem = (int)sizeof(OutSmem<kR>);
  const cudaError_t e = cudaFuncSetAttribute(
      lin_out_kernel<T, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof_scope("kda_linear_out", s);
  return launch_chained(lin_out_kernel<T, kR>, dim3((unsigned)chunks, (unsigned)H, C / kR),
                        kOutThreads, smem, s, static_cast<const T*>(q), static_cast<const T*>(k),
                        static_cast<const T*>(v), g, g_head, scale, plan, H, Hk, states,
                        static_cast<T*>(o));
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
  int sms = 152, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (n_tokens > 0) {
    e = launch_local<T>(k, v, g, g_head, plan, chunks, H, Hk, local, gam, s);
    if (e != cudaSuccess) return e;
  }
  {
    ProfScope prof_scope("kda_linear_scan", s);
    e = launch_chained(lin_scan_kernel,
                       dim3((unsigned)((int64_t)n_seqs * H), D * D / 4 / kScanThreads),
                       kScanThreads, 0, s, h0, plan, H, local, gam, hT);
    if (e != cudaSuccess) return e;
  }
  if (n_tokens == 0) return cudaSuccess;
  // Few chunks and heads: the rows of a chunk are spread over four CTAs, each of which reads
  // all of its keys, state and values, while all of them run at once, two an SM (whole pass,
  // kR = 64 -> 16, by chunks x heads: 2 x 1 29.1 -> 21.8 us, 2 x 16 30.1 -> 23.5, 2 x 38 32.2 ->
  // 28.8, but 6 x 16 34.2 -> 37.8, 9 x 16 34.7 -> 43.0).
  if (2 * chunks * H <= sms)
    return launch_out<T, 16>(q, k, v, g, g_head, scale, plan, chunks, H, Hk, local, o, s);
  return launch_out<T, 64>(q, k, v, g, g_head, scale, plan, chunks, H, Hk, local, o, s);
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
