// kda_scan.cu -- selective state space scan over packed sequences: for every channel c with
// states s = 0 .. S-1 (S = 8, 16, 32) and delta_t = softplus(dt_t + bias),
//     h_t[s] = exp(delta_t A[s]) h_{t-1}[s] + delta_t x_t B_t[s]
//     y_t    = (sum_s C_t[s] h_t[s] + D x_t) SiLU(z_t)
// B and C are shared by the channels of a group.  The states are fp32.
//
// A CTA takes 256 / S neighbouring channels of one sequence.  Its warps take tiles of 8 tokens in
// turn and pass the state round: what a tile needs no state for (its inputs, the steps, the
// decays: one exponential a state, token and channel) is done ahead by all warps at once, and
// a warp that gets the state runs its 8 tokens, hands it on, and forms its outputs behind that.
// A lane holds 8 states of one channel (S / 8 lanes share a channel), the decays of the tile in
// registers; B, C and the steps come from shared memory.
#include <algorithm>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kScanWarps = 4;
constexpr int kTok = 8;  // tokens of a tile

__device__ __forceinline__ void copy16(uint32_t to, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // (0: zeros are written)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
// The state is handed from warp to warp through named barriers of the two (ids 1 ..).
__device__ __forceinline__ void handed(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void hand(int id) {
  asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

template <typename T, int kS>
struct ScanWarp {  // shared memory of a warp
  static constexpr int kLn = kS / 8, kCh = 32 / kLn;
  static constexpr int kPitch = kCh * (int)sizeof(T) + 16;  // (rows of lanes that read together
                                                            // lie in different banks)
  __align__(16) char raw[3][kTok][kPitch];  // x, dt, z as they lie in memory
  __align__(16) char bc[2][kTok][kS * sizeof(T)];
  __align__(16) float2 step[kTok][kCh];     // delta, delta x
  __align__(16) float BC[2][kTok][kS];
  __align__(16) float4 state[2][32];        // what the warp hands on
};

template <typename T, int kS>
__global__ void __launch_bounds__(32 * kScanWarps, 16 / kScanWarps) scan_kernel(const ScanArgs a, int* err) {
  using W = ScanWarp<T, kS>;
  constexpr int kLn = W::kLn, kCh = W::kCh, kMine = kTok / kLn;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  W& w = reinterpret_cast<W*>(smem)[warp];
  const int from = (warp + kScanWarps - 1) % kScanWarps;
  const W& before = reinterpret_cast<W*>(smem)[from];

  const int per_group = a.C / a.G;
  const int blocks = (per_group + kCh - 1) / kCh;  // of a group
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / ((int64_t)blocks * a.G));
  const int rest = (int)(unit - (int64_t)n * blocks * a.G);
  const int g = rest / blocks, first = (rest - g * blocks) * kCh;  // first channel in the group
  int64_t t0, t1;
  if (!seq_range(a, n, t0, t1) && threadIdx.x == 0 && err) atomicExch(err, kDevErrBadSeqlens);
  const int cl = lane % kCh, sub = lane / kCh;
  const int width = min(kCh, per_group - first);  // channels there are (a multiple of 8)
  const bool on = cl < width;
  const int c0 = g * per_group + first, c = c0 + (on ? cl : 0);
  const float bias = a.bias ? __ldg(a.bias + c) : 0.f, skip = a.D ? __ldg(a.D + c) : 0.f;
  float2 A[4];
  {
    float v[8];
    load8(a.A + (int64_t)c * kS + 8 * sub, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] = make_float2(kLog2e * v[2 * i], kLog2e * v[2 * i + 1]);
  }
  const int64_t at = ((int64_t)n * a.C + c) * kS + 8 * sub;

  // Copies of a tile: rows of x, dt and z by 16-byte pieces, then those of B and C.  A lane copies
  // the same pieces of every tile of its warp.
  constexpr int kRow = kCh * (int)sizeof(T) / 16, kBc = kS * (int)sizeof(T) / 16;
  constexpr int kX = kTok * kRow, kB = kTok * kBc;
  constexpr uint32_t kNone = ~0u;
  constexpr int kXs = (3 * kX + 31) / 32, kBs = (2 * kB + 31) / 32;
  const char* src[kXs + kBs];
  int64_t step[kXs + kBs];
  uint32_t to[kXs + kBs];  // (kNone: no piece)
  int row[kXs + kBs];      // (kTok: a piece behind the last channel)
#pragma unroll
  for (int k = 0; k < kXs + kBs; ++k) {
    const bool isx = k < kXs;
    const int p = 32 * (isx ? k : k - kXs) + lane;
    const int of = isx ? kX : kB, per = isx ? kRow : kBc;
    const int which = p / of, col = p % per;
    row[k] = p % of / per;
    const void* base = isx ? (which == 0 ? a.x : which == 1 ? a.dt : a.z) : which == 0 ? a.B : a.Cm;
    const int64_t stride = isx ? (which == 0 ? a.sx : which == 1 ? a.sdt : a.sz)
                               : which == 0 ? a.sB : a.sC;
    to[k] = p >= (isx ? 3 : 2) * of || !base ? kNone
            : (uint32_t)__cvta_generic_to_shared(isx ? &w.raw[which % 3][row[k]][16 * col]
                                                     : &w.bc[which % 2][row[k]][16 * col]);
    if (to[k] == kNone) base = a.x;
    const bool in = !isx || col * 16 / (int)sizeof(T) < width;
    src[k] = static_cast<const char*>(base) +
             ((t0 + (int64_t)warp * kTok + row[k]) * stride + (isx ? c0 : g * kS)) * (int)sizeof(T) +
             (in ? 16 * col : 0);
    step[k] = stride * kTok * kScanWarps * (int)sizeof(T);
    if (!in) row[k] = kTok;
  }
  // `left`: tokens of the sequence from the tile's first on
  auto fetch = [&](int left) {
#pragma unroll
    for (int k = 0; k < kXs + kBs; ++k) {
      if (to[k] != kNone) copy16(to[k], row[k] < left ? src[k] : static_cast<const char*>(a.x), row[k] < left && row[k] < kTok);
      src[k] += step[k];
    }
  };

  const int len = (int)(t1 - t0), tiles = (len + kTok - 1) / kTok;
  if (tiles == 0) {
    if (warp == 0 && a.hT && on) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a.h0 ? a.h0[at + i] : 0.f;
      store8(a.hT + at, v);
    }
    return;
  }
  if (warp < tiles) fetch(len - warp * kTok);
  T* y = static_cast<T*>(a.y) + (t0 + warp * kTok + kMine * sub) * a.sy + c;
  for (int tile = warp; tile < tiles; tile += kScanWarps, y += kScanWarps * kTok * a.sy) {
    const int left = len - tile * kTok - kMine * sub;  // tokens from the lane's own ones on
    wait_copies();
    __syncwarp();
    // steps, each by one lane; B and C to fp32
    float2 x[kMine / 2], z[kMine / 2];
#pragma unroll
    for (int j = 0; j < kMine / 2; ++j) {
      const int t = kMine * sub + 2 * j;
      auto two = [&](int which) {
        return make_float2(to_f32(reinterpret_cast<const T*>(w.raw[which][t])[cl]),
                           to_f32(reinterpret_cast<const T*>(w.raw[which][t + 1])[cl]));
      };
      x[j] = two(0);
      if (a.z) z[j] = two(2);
      float2 d = __fadd2_rn(two(1), both(bias));
      if (a.softplus) d = softplus2(d);
      if (2 * j >= left) d.x = 0.f;  // behind the end: the state stays
      if (2 * j + 1 >= left) d.y = 0.f;
      const float2 dx = __fmul2_rn(d, x[j]);
      w.step[t][cl] = make_float2(d.x, dx.x);
      w.step[t + 1][cl] = make_float2(d.y, dx.y);
    }
#pragma unroll
    for (int k = 0; k < (2 * kTok * kS / 8 + 31) / 32; ++k) {
      const int p = 8 * (32 * k + lane);
      if (p < 2 * kTok * kS) {
        float v[8];
        load8(reinterpret_cast<const T*>(w.bc) + p, v);
        store8(&w.BC[0][0][0] + p, v);
      }
    }
    __syncwarp();
    if (tile + kScanWarps < tiles) fetch(len - (tile + kScanWarps) * kTok);

    float2 e[kTok][4];  // the decays, then the states
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const float d = w.step[t][cl].x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = __fmul2_rn(A[i], make_float2(d, d));
        e[t][i] = make_float2(ex2(u.x), ex2(u.y));
      }
    }
    float2 h[4];
    if (tile == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = a.h0 ? *reinterpret_cast<const float2*>(a.h0 + at + 2 * i) : make_float2(0.f, 0.f);
    } else {
      handed(1 + from);
      const float4 lo = before.state[0][lane], hi = before.state[1][lane];
      h[0] = make_float2(lo.x, lo.y); h[1] = make_float2(lo.z, lo.w);
      h[2] = make_float2(hi.x, hi.y); h[3] = make_float2(hi.z, hi.w);
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const float dx = w.step[t][cl].y;
      const float4 lo = *reinterpret_cast<const float4*>(&w.BC[0][t][8 * sub]);
      const float4 hi = *reinterpret_cast<const float4*>(&w.BC[0][t][8 * sub + 4]);
      const float2 d2 = make_float2(dx, dx);
      e[t][0] = h[0] = __ffma2_rn(e[t][0], h[0], __fmul2_rn(d2, make_float2(lo.x, lo.y)));
      e[t][1] = h[1] = __ffma2_rn(e[t][1], h[1], __fmul2_rn(d2, make_float2(lo.z, lo.w)));
      e[t][2] = h[2] = __ffma2_rn(e[t][2], h[2], __fmul2_rn(d2, make_float2(hi.x, hi.y)));
      e[t][3] = h[3] = __ffma2_rn(e[t][3], h[3], __fmul2_rn(d2, make_float2(hi.z, hi.w)));
    }
    if (tile + 1 < tiles) {
      w.state[0][lane] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
      w.state[1][lane] = make_float4(h[2].x, h[2].y, h[3].x, h[3].y);
      hand(1 + warp);
    } else if (a.hT && on) {
      const float v[8] = {h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
      store8(a.hT + at, v);
    }
    float acc[kTok];
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const float4 lo = *reinterpret_cast<const float4*>(&w.BC[1][t][8 * sub]);
      const float4 hi = *reinterpret_cast<const float4*>(&w.BC[1][t][8 * sub + 4]);
      float2 s = __fmul2_rn(e[t][0], make_float2(lo.x, lo.y));
      s = __ffma2_rn(e[t][1], make_float2(lo.z, lo.w), s);
      s = __ffma2_rn(e[t][2], make_float2(hi.x, hi.y), s);
      s = __ffma2_rn(e[t][3], make_float2(hi.z, hi.w), s);
      acc[t] = s.x + s.y;
    }
    // halving exchange inside a channel's lanes: lane sub ends with tokens kMine sub ..
#pragma unroll
    for (int m = kLn / 2, keep = kTok / 2; m > 0; m /= 2, keep /= 2) {
      const bool upper = (sub & m) != 0;
#pragma unroll
      for (int j = 0; j < keep; ++j) {
        const float other = __shfl_xor_sync(0xffffffffu, upper ? acc[j] : acc[j + keep], m * kCh);
        acc[j] = (upper ? acc[j + keep] : acc[j]) + other;
      }
    }
#pragma unroll
    for (int j = 0; j < kMine / 2; ++j) {
      float2 v = __ffma2_rn(both(skip), x[j], make_float2(acc[2 * j], acc[2 * j + 1]));
      if (a.z) v = __fmul2_rn(v, silu2(z[j]));
      if (on && 2 * j < left) y[2 * j * a.sy] = from_f32<T>(v.x);
      if (on && 2 * j + 1 < left) y[(2 * j + 1) * a.sy] = from_f32<T>(v.y);
    }
    __syncwarp();  // step and BC may be written again
  }
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, int bf16, int S, int* err, cudaStream_t s) {
  const int ch = 256 / S;
  const int64_t units = (int64_t)a.N * a.G * ((a.C / a.G + ch - 1) / ch);
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_scan", s);
  cudaError_t e = cudaSuccess;
  with_states(S, [&](auto k) {
    constexpr int kS = decltype(k)::value;
    auto launch = [&](auto kernel, size_t smem) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e == cudaSuccess)
        kernel<<<(unsigned)units, 32 * kScanWarps, smem, s>>>(a, err);
    };
    if (bf16)
      launch(scan_kernel<__nv_bfloat16, kS>, kScanWarps * sizeof(ScanWarp<__nv_bfloat16, kS>));
    else
      launch(scan_kernel<float, kS>, kScanWarps * sizeof(ScanWarp<float, kS>));
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
