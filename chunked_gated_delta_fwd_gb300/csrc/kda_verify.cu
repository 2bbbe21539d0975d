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
// and then across the cluster; the warp whose piece the limit falls into looks it through again,
// by lanes' runs and then token by token.
//
// Bound by HBM for large batches (one row of p, one of q where a token was rejected) and by its
// chain of loads for small ones: drafted token -> its probabilities -> rows -> search.  128 rows of
// 163840: fp32 31 to 35 us (4.3 to 4.8 TB/s of the rows it needs), bf16 21 to 24 us; of 163841, whose
// rows begin anywhere, token by token: 35 to 38 and 32 to 34 us (42 and 40 with 4 loads in flight); one
// row of 32000: 6 to 7 us, of 163840: 8 to 10.
#include <cooperative_groups.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

// A weight w in [0, 1] as a whole number of 2^-56, the rest cut off, in three parts of 23, 23 and
// 10 bits: w + 1 rounded down holds floor(2^23 w) in its low bits, and what is left of w, 2^23
// times as large, is taken the same way; what then is left, r < 2^-23, meets 2^-10, whose last bit
// is 2^-33: floor(2^33 r).  Every step is exact but for the cutting.  (In packed fp32
// and 32-bit sums: a conversion to 64 bits takes a clock an SM, 74 us for 128 rows of 163840 whose
// traffic takes 22; shifts of 64 bits 44 us.)
struct Parts {
  uint32_t hi, mid, lo;  // sums of the parts with the exponent's bits of what held them
};
constexpr uint32_t kOne = 0x3f800000u, kLast = 0x3a800000u;  // 1.f and 2^-10
__device__ __forceinline__ void add_pair(Parts& s, float w0, float w1) {
  const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
  const float2 scale = make_float2(0x1p23f, 0x1p23f), neg = make_float2(-0x1p23f, -0x1p23f);
  const float2 w = make_float2(w0, w1);
  const float2 t1 = __fadd2_rz(w, one);
  // 2^23 (w - (t1 - 1)) = (2^23 w + 2^23) - 2^23 t1, in an order whose steps are exact
  const float2 r1 = __ffma2_rn(__fadd2_rn(t1, minus), neg, __fmul2_rn(w, scale));
  const float2 t2 = __fadd2_rz(r1, one);
  const float2 r2 = __ffma2_rn(__fadd2_rn(t2, minus), minus, r1);
  const float2 t3 = __fadd2_rz(r2, make_float2(0x1p-10f, 0x1p-10f));
  s.hi += __float_as_uint(t1.x) + __float_as_uint(t1.y);
  s.mid += __float_as_uint(t2.x) + __float_as_uint(t2.y);
  s.lo += __float_as_uint(t3.x) + __float_as_uint(t3.y);
}
// The sum of n <= 511 weights added up in s.
__device__ __forceinline__ uint64_t total_of(const Parts& s, uint32_t n) {
  return ((uint64_t)(s.hi - n * kOne) << 33) + ((uint64_t)(s.mid - n * kOne) << 10) +
         (s.lo - n * kLast);
}
__device__ __forceinline__ uint64_t units_of(float w) {
  Parts s{0, 0, 0};
  add_pair(s, w, 0.f);
  return total_of(s, 2);
}

// p - q, held to [0, 1]; what is not a number is 0.
__device__ __forceinline__ float left_of(float p, float q) { return __saturatef(__fsub_rn(p, q)); }

// The weight of token v: of p, or of what is left of it behind q.
template <typename T>
__device__ __forceinline__ uint64_t weight(const T* p, const T* q, int64_t v) {
  return units_of(left_of(to_f32(p[v]), q ? to_f32(q[v]) : 0.f));
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

// The halves of a cluster's barrier.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// The first lane whose running sum passes the limit (one does).
__device__ __forceinline__ int first_over(uint64_t upto, uint64_t limit) {
  return (__ffs((int)__ballot_sync(kAll, upto > limit)) - 1) & 31;
}
// What comes before entry i of an inclusive scan over the lanes.
__device__ __forceinline__ uint64_t exclusive(uint64_t upto, int i) {
  const uint64_t x = __shfl_sync(kAll, upto, (i + 31) & 31);
  return i > 0 ? x : 0;
}

// Sum of the weights of tokens [begin, end) over the warp, every lane its share.
template <typename T, bool kVec, bool kQ>
__device__ __forceinline__ uint64_t lane_sum(const T* p, const T* q, int64_t begin, int64_t end,
                                             int lane) {
  constexpr int kN = kVec ? 16 / (int)sizeof(T) : 1;
  // Loads of a lane in flight: 16 tokens; 8 of fp32 one by one (whose registers are as many).
  constexpr int kAhead = kVec || sizeof(T) == 2 ? 16 / kN : 8;
  uint64_t sum = 0;
  for (int64_t v0 = begin; v0 < end; v0 += 32 * kN * kAhead) {
    float x[kAhead][kN], y[kAhead][kN];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t v = v0 + kN * (32 * i + lane);
#pragma unroll
      for (int j = 0; j < kN; ++j) x[i][j] = y[i][j] = 0.f;
      if (v >= end) continue;
      if constexpr (kVec) {
        if constexpr (sizeof(T) == 2) load8(p + v, x[i]); else load4(p + v, x[i]);
        if constexpr (kQ) {
          if constexpr (sizeof(T) == 2) load8(q + v, y[i]); else load4(q + v, y[i]);
        }
      } else {
        x[i][0] = to_f32(p[v]);
        if constexpr (kQ) y[i][0] = to_f32(q[v]);
      }
    }
    Parts part{0, 0, 0};
#pragma unroll
    for (int i = 0; i < kAhead * kN; i += 2)
      add_pair(part, left_of(x[i / kN][i % kN], kQ ? y[i / kN][i % kN] : 0.f),
               left_of(x[(i + 1) / kN][(i + 1) % kN], kQ ? y[(i + 1) / kN][(i + 1) % kN] : 0.f));
    sum = add(sum, total_of(part, kAhead * kN));
  }
  return sum;
}

// kVec: rows begin on 16-byte boundaries and hold whole 16-byte pieces.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(
    const int32_t* __restrict__ draft, const T* __restrict__ q, const T* __restrict__ p,
    const float* __restrict__ u_accept, const float* __restrict__ u_sample,
    int32_t* __restrict__ tokens, int32_t* __restrict__ n_advance, int Tn, int V, int per, int share) {
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

  const int64_t begin = min((int64_t)V, (rank * kVerifyWarps + warp) * (int64_t)per);
  const int64_t end = min((int64_t)V, begin + per);
  uint64_t total = 0, before = 0, mine = 0, upto = 0, cta_before = 0;
  for (;;) {
    mine = warp_sum(qr ? lane_sum<T, kVec, true>(pr, qr, begin, end, lane)
                       : lane_sum<T, kVec, false>(pr, nullptr, begin, end, lane));
    if (lane == 0) piece[warp] = mine;
    __syncthreads();
    upto = warp_inclusive(lane < kVerifyWarps ? piece[lane] : 0, lane);  // over the CTA's pieces
    if (threadIdx.x == 31) cta_total = upto;
    __syncwarp();
    cluster.sync();
    const uint64_t y = lane < ctas ? *cluster.map_shared_rank(&cta_total, lane) : 0;
    const uint64_t to_cta = warp_inclusive(y, lane);
    total = __shfl_sync(kAll, to_cta, 31);
    cta_before = exclusive(to_cta, rank);
    cluster_arrive();  // this CTA has read the others' sums
    if (total > 0 || !qr) break;
    cluster_wait();
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
  if (limit >= cta_before && limit < add(cta_before, cta_total)) {
    // the piece that passes the limit, shared by this CTA's warps, a part each
    const int hit = first_over(add(cta_before, upto), limit);
    before = add(cta_before, exclusive(upto, hit));
    const int64_t base = ((int64_t)rank * kVerifyWarps + hit) * per;
    const int64_t stop = min((int64_t)V, base + per);
    const int64_t part = base + (int64_t)warp * share, part_end = min(stop, part + share);
    mine = warp_sum(qr ? lane_sum<T, kVec, true>(pr, qr, part, part_end, lane)
                       : lane_sum<T, kVec, false>(pr, nullptr, part, part_end, lane));
    __syncthreads();  // everyone has read the pieces' sums
    if (lane == 0) piece[warp] = mine;
    __syncthreads();
    upto = add(before, warp_inclusive(lane < kVerifyWarps ? piece[lane] : 0, lane));
    const int owner = first_over(upto, limit);
    if (warp == owner) {
      // a run of consecutive tokens a lane, and of the run that passes the limit token by token
      const int run = (share + 31) / 32;
      before = owner > 0 ? __shfl_sync(kAll, upto, (owner + 31) & 31) : before;
      const int64_t from = part + (int64_t)lane * run, to = min(part_end, from + run);
      uint64_t sum = 0;
#pragma unroll 8
      for (int64_t v = from; v < to; ++v) sum = add(sum, weight(pr, qr, v));
      upto = add(before, warp_inclusive(sum, lane));
      const int in = first_over(upto, limit);
      before = in > 0 ? __shfl_sync(kAll, upto, (in + 31) & 31) : before;
      const int64_t first = part + (int64_t)in * run, last = min(part_end, first + run);
      for (int64_t v0 = first; v0 < last; v0 += 32) {
        const int64_t v = v0 + lane;
        upto = add(before, warp_inclusive(v < last ? weight(pr, qr, v) : 0, lane));
        const unsigned over = __ballot_sync(kAll, upto > limit);
        if (over) {
          if (lane == 0) out[k] = (int32_t)(v0 + __ffs((int)over) - 1);
          break;
        }
        before = __shfl_sync(kAll, upto, 31);
      }
    }
  }
  cluster_wait();  // the others have read this CTA's sum
}

}  // namespace

cudaError_t launch_verify(const int32_t* draft, const void* q, const void* p, int bf16,
                          const float* u_accept, const float* u_sample, int32_t* tokens,
                          int32_t* n_advance, int N, int T, int V, cudaStream_t s) {
  ProfScope prof_scope("kda_verify", s);
  int ctas = kMaxCluster;
  // Half the CTAs a sequence where the others would have a load of 128 tokens a warp or none, or
  // where the batch fills the SMs twice over without them (128 rows of 163840 fp32: 44 us with 8,
  // 35 with 4, 31 with 2, 39 with 1; one row: 7.8, 8.6, 12, 16).
  while (ctas > 1 && (V <= ctas / 2 * kVerifyWarps * 128 || (int64_t)N * ctas > 304)) ctas /= 2;
  const int whole = bf16 ? 8 : 4;  // tokens of a 16-byte piece
  const bool vec = V % whole == 0;
  const int64_t step = vec ? 32 * whole : 32, warps = (int64_t)ctas * kVerifyWarps;
  const int per = (int)((((int64_t)V + warps - 1) / warps + step - 1) / step * step);
  const int share = (int)(((per + kVerifyWarps - 1) / kVerifyWarps + step - 1) / step * step);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(N * ctas));
  c.blockDim = dim3(kVerifyThreads);
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  if (bf16) {
    const auto* pq = static_cast<const __nv_bfloat16*>(q);
    const auto* pp = static_cast<const __nv_bfloat16*>(p);
    return vec ? cudaLaunchKernelEx(&c, verify_kernel<__nv_bfloat16, true>, draft, pq, pp, u_accept,
                                    u_sample, tokens, n_advance, T, V, per, share)
               : cudaLaunchKernelEx(&c, verify_kernel<__nv_bfloat16, false>, draft, pq, pp, u_accept,
                                    u_sample, tokens, n_advance, T, V, per, share);
  }
  const auto* pq = static_cast<const float*>(q);
  const auto* pp = static_cast<const float*>(p);
  return vec ? cudaLaunchKernelEx(&c, verify_kernel<float, true>, draft, pq, pp, u_accept, u_sample,
                                  tokens, n_advance, T, V, per, share)
             : cudaLaunchKernelEx(&c, verify_kernel<float, false>, draft, pq, pp, u_accept, u_sample,
                                  tokens, n_advance, T, V, per, share);
}

}  // namespace kda
