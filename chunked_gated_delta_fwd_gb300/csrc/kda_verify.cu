// kda_verify.cu -- verification of drafted tokens against the target's probabilities.  Of the
// drafted d_0 .. d_{T-1}, d_i drawn from q_i, with given uniform numbers u_i and u:
//     d_i is accepted while u_i q_i(d_i) < p_i(d_i);
// behind the k accepted ones a token is drawn, from max(p_k - q_k, 0) where d_k was rejected and
// from p_k where the draft had ended: the first v with w_0 + .. + w_v > u (w_0 + .. + w_{V-1}).
//
// The products are exact in 64 bits and the weights are whole numbers of 2^-56 (the difference
// rounded to fp32 before, which moves a weight by 2^-24 of itself), so the sums are exact:
// they do not depend on how the row is split, and no border is decided by an order of additions.
//
// A cluster of CTAs shares a sequence.  Every warp finds the accepted count by itself (T loads
// side by side), sums one contiguous piece of the row, and the pieces' sums meet in shared memory
// and then across the cluster; the warp whose piece the limit falls into looks it through again.
#include <cooperative_groups.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

// A probability as a whole number of 2^-56; what is not above 0 (NaN too) weighs nothing.
__device__ __forceinline__ uint64_t units_of(float w) {
  return __float2ull_rz(fminf(fmaxf(w, 0.f), 1.f) * 0x1p56f);
}

template <typename T>
__device__ __forceinline__ uint64_t weight(const T* p, const T* q, int64_t v) {
  float w = to_f32(p[v]);
  if (q) w = __fsub_rn(w, to_f32(q[v]));
  return units_of(w);
}

// Sums stop at 2^64 - 1 (weights that add up to 256 or more), in any order: a running sum always
// reaches the total, so that there is a first v in any case.
__device__ __forceinline__ uint64_t add(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  return s < a ? ~0ull : s;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = add(x, __shfl_xor_sync(kAll, x, o));
  return x;
}
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x = add(x, y);
  }
  return x;
}

// What comes before entry i of an inclusive scan over the lanes.
__device__ __forceinline__ uint64_t exclusive(uint64_t upto, int i) {
  const uint64_t x = __shfl_sync(kAll, upto, (i + 31) & 31);
  return i > 0 ? x : 0;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(
    const int32_t* __restrict__ draft, const T* __restrict__ q, const T* __restrict__ p,
    const float* __restrict__ u_accept, const float* __restrict__ u_sample,
    int32_t* __restrict__ tokens, int32_t* __restrict__ n_advance, int Tn, int V) {
  __shared__ uint64_t piece[kVerifyWarps];
  __shared__ uint64_t cta_total;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t n = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  bool ok = false, real = false;
  int32_t d = -1;
  if (lane < Tn) {
    d = __ldg(draft + n * Tn + lane);
    real = d >= 0 && d < V;
    if (real) {
      const float pd = to_f32(p[(n * (Tn + 1) + lane) * V + d]);
      const float qd = to_f32(q[(n * Tn + lane) * V + d]);
      ok = (double)__ldg(u_accept + n * Tn + lane) * (double)qd < (double)pd;
    }
  }
  const int k = __ffs((int)~__ballot_sync(kAll, ok)) - 1;  // (lane Tn is never ok)
  const bool rejected = __shfl_sync(kAll, (int)real, k) != 0;
  const T* pr = p + (n * (Tn + 1) + k) * V;
  const T* qr = rejected ? q + (n * Tn + k) * V : nullptr;

  const int64_t per = (V + (int64_t)ctas * kVerifyWarps - 1) / ((int64_t)ctas * kVerifyWarps);
  const int64_t begin = min((int64_t)V, (rank * kVerifyWarps + warp) * per);
  const int64_t end = min((int64_t)V, begin + per);
  uint64_t total = 0, before = 0, mine = 0;
  for (;;) {
    uint64_t sum = 0;
    for (int64_t v = begin + lane; v < end; v += 32) sum = add(sum, weight(pr, qr, v));
    mine = warp_sum(sum);
    if (lane == 0) piece[warp] = mine;
    __syncthreads();
    const uint64_t x = lane < kVerifyWarps ? piece[lane] : 0;
    const uint64_t upto = warp_inclusive(x, lane);
    before = exclusive(upto, warp);
    if (threadIdx.x == 31) cta_total = upto;
    cluster.sync();
    const uint64_t y = lane < ctas ? *cluster.map_shared_rank(&cta_total, lane) : 0;
    const uint64_t to_cta = warp_inclusive(y, lane);
    total = __shfl_sync(kAll, to_cta, 31);
    before = add(exclusive(to_cta, rank), before);
    cluster.sync();  // the sums may be written again, or their CTA may end
    if (total > 0 || !qr) break;
    qr = nullptr;  // nothing is left of p behind q: p itself
  }
  const float u = __ldg(u_sample + n);
  const uint64_t uu = __float2ull_rz(fminf(fmaxf(u, 0.f), 1.f - 0x1p-24f) * 0x1p24f);
  const uint64_t limit = (__umul64hi(total, uu) << 40) | ((total * uu) >> 24);
  int32_t* out = tokens + n * (Tn + 1);
  if (rank == 0 && warp == 0) {
    if (lane < Tn + 1 && lane != k) out[lane] = lane < k ? d : -1;
    if (lane == 0) n_advance[n] = k + 1;
    if (lane == 0 && total == 0) out[k] = 0;
  }
  if (limit < before || limit >= add(before, mine)) return;
  for (int64_t v0 = begin; v0 < end; v0 += 32) {
    const int64_t v = v0 + lane;
    const uint64_t w = v < end ? weight(pr, qr, v) : 0;
    const uint64_t upto = add(before, warp_inclusive(w, lane));
    const unsigned over = __ballot_sync(kAll, upto > limit);
    if (over) {
      if (lane == 0) out[k] = (int32_t)(v0 + __ffs((int)over) - 1);
      return;
    }
    before = __shfl_sync(kAll, upto, 31);
  }
}

}  // namespace

cudaError_t launch_verify(const int32_t* draft, const void* q, const void* p, int bf16,
                          const float* u_accept, const float* u_sample, int32_t* tokens,
                          int32_t* n_advance, int N, int T, int V, cudaStream_t s) {
  ProfScope prof_scope("kda_verify", s);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)N * kMaxCluster);
  c.blockDim = dim3(kVerifyThreads);
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kMaxCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  if (bf16)
    return cudaLaunchKernelEx(&c, verify_kernel<__nv_bfloat16>, draft,
                              static_cast<const __nv_bfloat16*>(q),
                              static_cast<const __nv_bfloat16*>(p), u_accept, u_sample, tokens,
                              n_advance, T, V);
  return cudaLaunchKernelEx(&c, verify_kernel<float>, draft, static_cast<const float*>(q),
                            static_cast<const float*>(p), u_accept, u_sample, tokens, n_advance, T, V);
}

}  // namespace kda
