// kda_linear_tc.cu -- the prompt pass of linear attention with a decay for each head,
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// for bf16 inputs on the sm_103a tensor cores.  In chunks of 128 tokens, G the running sum
// of g inside the chunk and S the state before it:
//     O_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//     S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// A decay is one number a token and head, so it scales rows and columns of the products
// in fp32 and no operand leaves the range of bf16, whatever g <= 0 is.
//
// One CTA per SM walks (sequence, head) chains chunk by chunk; the state stays in tensor
// memory as S^T (lanes = value rows, fp32) for a whole chain.  Four MMA groups a chunk
// (M = N = K = 128 each):
//     QK   scores = Q K^T                      (lanes = tokens)
//     QS   Q S, from a bf16 copy of S^T        (lanes = tokens)
//     KV   S^T += V^T Kw, Kw_j = e^{G_C - G_j} k_j, after S^T *= e^{G_C}
//     PV   P V with P = scale * decay * scores, bf16, from tensor memory
// QS and PV have an accumulator each: e^{G_i} is applied to Q S in fp32 where o is written.
// Rounding: P and the copy of S to bf16 (o is bf16 as well, each adds an error of the size
// of o's own rounding).  The final state is fp32, so Kw is kept as two bf16 parts, hi + lo
// (16 bits of each weighted key), and KV is issued for both.
//
// Tiles of q, k and v arrive by tensor copies, 128-byte swizzled; the same bytes serve as a
// K-major operand (channels contracted) and as an MN-major one (tokens contracted), so
// nothing is transposed.  Kw overwrites the k tile in place (hi) and one more tile (lo).
//
// Warps: copy, MMA issue, decay vectors; then four groups of four, one warp of each on
// every SM sub-partition: weighted keys, scores -> P, outputs, state.
//
// Decays.  With L_i the sum of g inside a 32-token block up to i, U_j the sum behind j in
// its block and T_b the block totals, every exponent but those inside a diagonal block is
// a sum of non-positive terms: e^{G_i - G_j} = e^{L_i + T between} e^{U_j}, so a decay is
// as exact as fp32 addition next to any g.  Inside a block it is e^{L_i - L_j}.  g is held
// at -100 at least (e^-100 is 0 in fp32), which also makes -inf drop the state.
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int C = 128;  // tokens of a chunk
constexpr int D = kD;   // 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinG = -100.f;

constexpr int kSlots = 5;                  // ring of q / k / v tiles
constexpr uint32_t kTileBytes = C * D * 2;  // 32 KB: two 64-channel blocks of 128 rows
constexpr uint32_t kHalfTile = kTileBytes / 2;
constexpr uint32_t kLoOff = kSlots * kTileBytes;
constexpr uint32_t kSbOff = kLoOff + kTileBytes;   // bf16 copy of S^T, K-major
constexpr uint32_t kVecOff = kSbOff + kTileBytes;  // two decay vectors
struct Vec {
  float L[C];   // sum of g (log2 units) inside the token's 32-token block, inclusive
  float cf[C];  // 2^(sum of g behind the token inside its block)
  float T[4];   // block totals
  float pad[4];
};
constexpr uint32_t kBarOff = kVecOff + 2 * sizeof(Vec);
constexpr uint32_t kSmemUsed = kBarOff + 24 * 8 + 16;
constexpr uint32_t kSmemBytes = 232448;  // all an SM has: one CTA each
static_assert(kSmemUsed <= kSmemBytes, "shared memory");

// barriers
enum {
  bFull = 0,              // [5] tile landed
  bEmpty = bFull + kSlots,  // [5] tile read by its last MMA
  bVFull = bEmpty + kSlots,  // [2] decay vector written
  bVEmpty = bVFull + 2,      // [2] decay vector read
  bQK = bVEmpty + 2,         // scores complete
  bKt = bQK + 1,             // [2] weighted keys of tokens 0-63, 64-127 written
  bP = bKt + 2,              // P written
  bS = bP + 1,               // state scaled and copied
  bKV = bS + 1,              // state updated
  bPV = bKV + 1,             // outputs complete
  bO = bPV + 1,              // accumulators read out
  bDrain = bO + 1,
  kBars = bDrain + 1
};
static_assert(kBars <= 24, "barriers");

constexpr uint32_t kT_S = 0, kT_P = 128, kT_QS = 256, kT_PV = 384;  // TMEM columns

constexpr int kGroup = 128;
constexpr int kThreads = 128 + 4 * kGroup;

struct LinArgs {
  const float* g;
  int g_head;
  float scale;
  const float* h0;
  const int32_t* cu;  // null: sequences of T tokens
  int64_t T, n_tokens;
  int n_seqs, H, rep;
  __nv_bfloat16* o;
  float* hT;
  // segments (null tab: a chain is a whole sequence)
  const int4* tab;      // per segment: sequence, first token, tokens, index (last: bit 31)
  const int* n_segs;
  const float* s_in;    // states entering segments [segment][H][dv][dk]
  float* s_end;         // local end states
  float* seg_decay;     // [segment][H]
  int* err;
};

struct Job {
  int h, tokens, chunks;
  int64_t t0;
  const float* init;
  float* fin;
  float* decay;
};

// Tokens of sequence n, clamped to the inputs; a malformed cu_seqlens is reported.
__device__ __forceinline__ void seq_range(const LinArgs& a, int n, int64_t& t0, int64_t& t1) {
  if (!a.cu) {
    t0 = (int64_t)n * a.T;
    t1 = t0 + a.T;
    return;
  }
  const int64_t x0 = __ldg(a.cu + n), x1 = __ldg(a.cu + n + 1);
  t0 = x0 < 0 ? 0 : (x0 > a.n_tokens ? a.n_tokens : x0);
  t1 = x1 > a.n_tokens ? a.n_tokens : x1;
  bool bad = x0 != t0 || x1 != t1 || t1 < t0 || (n == 0 && x0 != 0) ||
             (n == a.n_seqs - 1 && x1 != a.n_tokens);
  if (t1 < t0) t1 = t0;
  if (bad && a.err) atomicExch(a.err, kDevErrBadSeqlens);
}

template <bool kOut>
__device__ __forceinline__ int job_count(const LinArgs& a) {
  return (a.tab ? __ldg(a.n_segs) : a.n_seqs) * a.H;
}

template <bool kOut>
__device__ __forceinline__ Job get_job(const LinArgs& a, int item) {
  Job j;
  const int u = item / a.H;
  j.h = item - u * a.H;
  j.decay = nullptr;
  if (!a.tab) {
    int64_t t1;
    seq_range(a, u, j.t0, t1);
    j.tokens = (int)(t1 - j.t0);
    const int64_t s = (int64_t)item * D * D;
    j.init = a.h0 ? a.h0 + s : nullptr;
    j.fin = a.hT ? a.hT + s : nullptr;
  } else {
    const int4 e = a.tab[u];
    j.t0 = e.y;
    j.tokens = e.z;
    const int k = e.w & 0x7fffffff;
    const bool last = e.w < 0;
    const int64_t sn = ((int64_t)e.x * a.H + j.h) * D * D, su = (int64_t)item * D * D;
    if (kOut) {
      j.init = a.s_in + su;
      j.fin = last && a.hT ? a.hT + sn : nullptr;
    } else {
      if (last) j.tokens = 0;  // nothing follows the last segment
      j.init = k == 0 && a.h0 ? a.h0 + sn : nullptr;
      j.fin = last ? nullptr : a.s_end + su;
      j.decay = a.seg_decay + item;
    }
  }
  j.chunks = (j.tokens + C - 1) / C;
  return j;
}

// kOut: outputs and final states.  Otherwise the state alone (the first pass over segments).
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    lin_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const LinArgs a) {
  constexpr int kTiles = kOut ? 3 : 2;  // tiles a chunk, in the order k, (q,) v
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  if (pad + kSmemUsed > kSmemBytes) {  // (uniform; dynamic shared memory starts aligned)
    if (threadIdx.x == 0 && a.err) atomicExch(a.err, kDevErrTimeout);
    return;
  }
  uint8_t* sm = smem_raw + pad;
  const uint32_t base = smem_addr(sm);
  const uint32_t bars = base + kBarOff;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBarOff + 24 * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kBarOff + 24 * 8 + 8);
  Vec* vecs = reinterpret_cast<Vec*>(sm + kVecOff);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

  if (t == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(bFull + i), 1);
      mbar_init(bar(bEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bVFull + i), 1);
      mbar_init(bar(bVEmpty + i), kOut ? 16 : 8);  // warps that read the vector
      mbar_init(bar(bKt + i), 4);
    }
    mbar_init(bar(bQK), 1);
    mbar_init(bar(bP), 4);
    mbar_init(bar(bS), 4);
    mbar_init(bar(bKV), 1);
    mbar_init(bar(bPV), 1);
    mbar_init(bar(bO), 4);
    mbar_init(bar(bDrain), 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 3) tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int items = job_count<kOut>(a);
  auto wait = [&](int b, uint32_t parity) {
    return wait_or_abort(bar(b), parity & 1u, a.err, abort_flag);
  };
  // the same for a whole warp: one outcome, so that warp-wide instructions stay together
  auto wait_warp = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(b, parity)) != 0;
  };
  // ring position of tile i of chunk `it` (0: k, then q with outputs, last: v)
  auto slot_of = [&](int it, int i) { return (kTiles * it + i) % kSlots; };
  auto phase_of = [&](int it, int i) { return (uint32_t)((kTiles * it + i) / kSlots) & 1u; };

  if (warp == 0) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      int m = 0;  // tiles issued
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Job j = get_job<kOut>(a, item);
        for (int c = 0; c < j.chunks && ok; ++c) {
          const int tok = (int)(j.t0 + (int64_t)c * C);
          for (int i = 0; i < kTiles; ++i, ++m) {
            const int s = m % kSlots;
            if (m >= kSlots && !wait(bEmpty + s, (uint32_t)(m / kSlots - 1))) {
              ok = false;
              break;
            }
            const bool is_v = i == kTiles - 1;
            const void* tm = is_v ? &tm_v : (i == 0 ? &tm_k : &tm_q);
            const int head = is_v ? j.h : j.h / a.rep;
            const uint32_t dst = base + s * kTileBytes;
            mbar_arrive_expect_tx(bar(bFull + s), kTileBytes);
            tma_load_3d(dst, tm, 0, head, tok, bar(bFull + s));
            tma_load_3d(dst + kHalfTile, tm, 64, head, tok, bar(bFull + s));
          }
        }
      }
      if (*abort_flag)  // copies in flight must land before the CTA exits
        for (int x = max(0, m - kSlots); x < m; ++x)
          mbar_wait(bar(bFull + x % kSlots), (uint32_t)(x / kSlots) & 1u, a.err);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------------- MMAs
    // Order a chunk: QS, KV, PV, then QK of the next chunk.  KV goes as early as its
    // operands allow: the state group works on its result while PV and QK run.
    if (lane == 0) {
      int total = 0;
      for (int item = blockIdx.x; item < items; item += gridDim.x)
        total += get_job<kOut>(a, item).chunks;
      const uint32_t id_kk = idesc_bf16_mn(C, C, 0, 0);  // both operands K-major
      const uint32_t id_kn = idesc_bf16_mn(C, D, 0, 1);  // B MN-major
      const uint32_t id_nn = idesc_bf16_mn(D, D, 1, 1);  // both MN-major
      bool any = false;
      auto tile = [&](int it, int i) { return base + (uint32_t)slot_of(it, i) * kTileBytes; };
      // K step s of a K-major tile / of an MN-major one (descriptors of step 0, advanced)
      auto kstep = [](int s) { return (uint32_t)(s >> 2) * kHalfTile + (uint32_t)(s & 3) * 32u; };
      auto qk = [&](int it) {
        if (!wait(bFull + slot_of(it, 0), phase_of(it, 0)) ||
            !wait(bFull + slot_of(it, 1), phase_of(it, 1)))
          return false;
        tc_fence_after();
        const uint64_t dq = kmajor_desc(tile(it, 1), C, 0), dk = kmajor_desc(tile(it, 0), C, 0);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_bf16(tmem + kT_P, desc_advance(dq, kstep(s)), desc_advance(dk, kstep(s)), id_kk, s > 0);
        mma_commit(bar(bQK));
        any = true;
        return true;
      };
      bool ok = total == 0 || !kOut || qk(0);
      for (int it = 0; it < total && ok; ++it) {
        const uint32_t par = (uint32_t)it;
        ok = wait(bS, par);
        if (!ok) break;
        if (kOut) {
          if (it > 0 && !wait(bO, par - 1)) break;
          tc_fence_after();
          const uint64_t dq = kmajor_desc(tile(it, 1), C, 0),
                         ds = kmajor_desc(base + kSbOff, D, 0);
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_bf16(tmem + kT_QS, desc_advance(dq, kstep(s)), desc_advance(ds, kstep(s)), id_kk,
                     s > 0);
          mma_commit(bar(bEmpty + slot_of(it, 1)));
          any = true;
        }
        ok = wait(bFull + slot_of(it, kTiles - 1), phase_of(it, kTiles - 1));
        const uint64_t dv = mnmajor_desc_lbo(tile(it, kTiles - 1), kHalfTile, 1024, 0);
        const uint64_t dhi = mnmajor_desc_lbo(tile(it, 0), kHalfTile, 1024, 0);
        const uint64_t dlo = mnmajor_desc_lbo(base + kLoOff, kHalfTile, 1024, 0);
        for (int hf = 0; hf < 2 && ok; ++hf) {  // tokens 0-63, 64-127
          ok = wait(bKt + hf, par);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < C / 32; ++s) {
            const uint32_t off = (uint32_t)(4 * hf + s) * 2048u;
            mma_bf16(tmem + kT_S, desc_advance(dv, off), desc_advance(dlo, off), id_nn, 1u);
            mma_bf16(tmem + kT_S, desc_advance(dv, off), desc_advance(dhi, off), id_nn, 1u);
          }
          any = true;
        }
        if (!ok) break;
        mma_commit(bar(bKV));
        mma_commit(bar(bEmpty + slot_of(it, 0)));
        if (kOut) {
          ok = wait(bP, par);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16_ta(tmem + kT_PV, tmem + kT_P + 8 * s, desc_advance(dv, (uint32_t)s * 2048u),
                        id_kn, s > 0);
          mma_commit(bar(bPV));
        }
        mma_commit(bar(bEmpty + slot_of(it, kTiles - 1)));
        if (kOut && it + 1 < total) ok = qk(it + 1);
      }
      if (*abort_flag && any) {  // drain MMAs in flight
        mma_commit(bar(bDrain));
        mbar_wait(bar(bDrain), 0, a.err);
      }
    }
  } else if (warp == 2) {
    // ----------------------------------------------------------- decay vectors
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const Job j = get_job<kOut>(a, item);
      for (int c = 0; c < j.chunks; ++c, ++it) {
        const int len = min(C, j.tokens - c * C);
        const int64_t tok = j.t0 + (int64_t)c * C;
        float g[4], u[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int r = 32 * b + lane;
          g[b] = 0.f;
          if (r < len) g[b] = __ldg(a.g + (a.g_head ? (int64_t)j.h : (tok + r) * a.H + j.h));
        }
        ok = it < 2 || wait_warp(bVEmpty + (it & 1), (uint32_t)(it >> 1) - 1);
        if (!ok) break;
        Vec& v = vecs[it & 1];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          g[b] = (g[b] < kMinG ? kMinG : g[b]) * kLog2e;  // NaN stays NaN
          u[b] = __shfl_down_sync(0xffffffffu, g[b], 1);
          if (lane == 31) u[b] = 0.f;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float x = __shfl_up_sync(0xffffffffu, g[b], o);
            const float y = __shfl_down_sync(0xffffffffu, u[b], o);
            if (lane >= o) g[b] += x;
            if (lane + o < 32) u[b] += y;
          }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          v.L[32 * b + lane] = g[b];
          v.cf[32 * b + lane] = exp2_approx(u[b]);
          if (lane == 31) v.T[b] = g[b];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bVFull + (it & 1)));
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ weighted keys
    // Two threads a row, 64 rows at a time: hi part in place, lo part into its own tile.
    // Rows past the sequence's end hold other tokens: their weighted keys and their
    // values become zeros, so that nothing of them (a NaN) meets this sequence.
    const int gt = t - 128, blk = gt & 1;
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const Job j = get_job<kOut>(a, item);
      for (int c = 0; c < j.chunks; ++c, ++it) {
        const int len = min(C, j.tokens - c * C);
        ok = wait_warp(bFull + slot_of(it, 0), phase_of(it, 0)) &&
             wait_warp(bVFull + (it & 1), (uint32_t)(it >> 1)) &&
             (!kOut || wait_warp(bQK, (uint32_t)it)) &&       // the raw keys are read
             (it == 0 || wait_warp(bKV, (uint32_t)it - 1)) &&  // the lo tile is read
             (len == C || wait_warp(bFull + slot_of(it, kTiles - 1), phase_of(it, kTiles - 1)));
        if (!ok) break;
        const Vec& v = vecs[it & 1];
        uint8_t* kt = sm + slot_of(it, 0) * kTileBytes + blk * kHalfTile;
        uint8_t* lo = sm + kLoOff + blk * kHalfTile;
        uint8_t* vt = sm + slot_of(it, kTiles - 1) * kTileBytes + blk * kHalfTile;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          const int r = 64 * hf + (gt >> 1), b = r >> 5;
          float after = 0.f;
#pragma unroll
          for (int x = 1; x < 4; ++x) after += x > b ? v.T[x] : 0.f;
          const float w = v.cf[r] * exp2_approx(after);
          const bool in = r < len;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint32_t off = (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
            const uint4 x = *reinterpret_cast<const uint4*>(kt + off);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = bf16_lo(xw[e]) * w, q = bf16_hi(xw[e]) * w;
              hw[e] = pack_bf16(p, q);
              lw[e] = pack_bf16(p - bf16_lo(hw[e]), q - bf16_hi(hw[e]));
              if (!in) hw[e] = lw[e] = 0u;
            }
            *reinterpret_cast<uint4*>(kt + off) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(lo + off) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            if (!in) *reinterpret_cast<uint4*>(vt + off) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(bKt + hf));
            if (hf == 1) mbar_arrive(bar(bVEmpty + (it & 1)));
          }
        }
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // -------------------------------------------------------------- scores -> P
    // Thread = token row.  P (packed pairs) overwrites the scores' columns from the left,
    // behind the block of scores being read.
    if (kOut) {
      const int w = warp & 3;
      const uint32_t row = tmem + ((uint32_t)(32 * w) << 16) + kT_P;
      int it = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Job j = get_job<kOut>(a, item);
        for (int c = 0; c < j.chunks; ++c, ++it) {
          ok = wait_warp(bVFull + (it & 1), (uint32_t)(it >> 1)) && wait_warp(bQK, (uint32_t)it);
          if (!ok) break;
          tc_fence_after();
          const Vec& v = vecs[it & 1];
          const float Li = v.L[32 * w + lane];
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t pk[16];
            if (b > w) {  // keys behind every token of this warp
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            } else {
              float s[32];
              tmem_ld32(row + 32 * b, s);
              tmem_wait_ld();
              if (b < w) {
                float between = 0.f;
#pragma unroll
                for (int x = 1; x < 3; ++x) between += (x > b && x < w) ? v.T[x] : 0.f;
                const float rf = a.scale * exp2_approx(Li + between);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 f = *reinterpret_cast<const float4*>(&v.cf[32 * b + i]);
                  pk[i / 2] = pack_bf16(s[i] * (f.x * rf), s[i + 1] * (f.y * rf));
                  pk[i / 2 + 1] = pack_bf16(s[i + 2] * (f.z * rf), s[i + 3] * (f.w * rf));
                }
              } else {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 L = *reinterpret_cast<const float4*>(&v.L[32 * b + i]);
                  const float Lj[4] = {L.x, L.y, L.z, L.w};
                  float p[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    p[e] = i + e <= lane ? s[i + e] * (a.scale * exp2_approx(Li - Lj[e])) : 0.f;
                  pk[i / 2] = pack_bf16(p[0], p[1]);
                  pk[i / 2 + 1] = pack_bf16(p[2], p[3]);
                }
              }
            }
            tmem_st16(row + 16 * b, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(bP));
            mbar_arrive(bar(bVEmpty + (it & 1)));
          }
        }
      }
    }
  } else if (warp >= 12 && warp < 16) {
    // ----------------------------------------------------------------- outputs
    if (kOut) {
      const int w = warp & 3, i0 = 32 * w + lane;
      const uint32_t row = tmem + ((uint32_t)(32 * w) << 16);
      int it = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Job j = get_job<kOut>(a, item);
        for (int c = 0; c < j.chunks; ++c, ++it) {
          const int len = min(C, j.tokens - c * C);
          ok = wait_warp(bVFull + (it & 1), (uint32_t)(it >> 1));
          if (!ok) break;
          const Vec& v = vecs[it & 1];
          float x = v.L[i0];
#pragma unroll
          for (int b = 0; b < 3; ++b) x += b < w ? v.T[b] : 0.f;
          const float E = a.scale * exp2_approx(x);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bVEmpty + (it & 1)));
          ok = wait_warp(bPV, (uint32_t)it);
          if (!ok) break;
          tc_fence_after();
          __nv_bfloat16* orow = a.o + ((j.t0 + (int64_t)c * C + i0) * a.H + j.h) * D;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            float qs[32], pv[32];
            tmem_ld32(row + kT_QS + 32 * p, qs);
            tmem_ld32(row + kT_PV + 32 * p, pv);
            tmem_wait_ld();
            if (p == 3) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(bO));
            }
            if (i0 < len) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t y[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                  y[f] = pack_bf16(fmaf(E, qs[e + 2 * f], pv[e + 2 * f]),
                                   fmaf(E, qs[e + 2 * f + 1], pv[e + 2 * f + 1]));
                *reinterpret_cast<uint4*>(orow + 32 * p + e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
      }
    }
  } else if (warp >= 16) {
    // ------------------------------------------------------------------- state
    // Thread = value row.  Before chunk c: the row to bf16 for QS (and times e^{G_C} back
    // into tensor memory for KV); the first chunk takes the initial state instead.
    const int dv = t - (128 + 3 * kGroup);
    const uint32_t row = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kT_S;
    uint8_t* sb = sm + kSbOff;
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const Job j = get_job<kOut>(a, item);
      float decay = 0.f;
      const float* init = j.init ? j.init + dv * D : nullptr;
      for (int c = 0; c < j.chunks; ++c, ++it) {
        ok = wait_warp(bVFull + (it & 1), (uint32_t)(it >> 1)) &&
             (c == 0 || wait_warp(bKV, (uint32_t)it - 1));
        if (!ok) break;
        tc_fence_after();
        const Vec& v = vecs[it & 1];
        const float tot = (v.T[0] + v.T[1]) + (v.T[2] + v.T[3]);
        decay += tot;
        const float gam = exp2_approx(tot);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float s[32];
          if (c > 0) {
            tmem_ld32(row + 32 * p, s);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 x = init ? *reinterpret_cast<const float4*>(init + 32 * p + i)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
              s[i] = x.x; s[i + 1] = x.y; s[i + 2] = x.z; s[i + 3] = x.w;
            }
          }
          if (kOut) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 y = make_uint4(pack_bf16(s[8 * e], s[8 * e + 1]),
                                         pack_bf16(s[8 * e + 2], s[8 * e + 3]),
                                         pack_bf16(s[8 * e + 4], s[8 * e + 5]),
                                         pack_bf16(s[8 * e + 6], s[8 * e + 7]));
              *reinterpret_cast<uint4*>(sb + sw128_chunk(D, dv, 4 * p + e)) = y;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] *= gam;
          tmem_st32(row + 32 * p, s);
        }
        tmem_wait_st();
        tc_fence_before();
        if (kOut) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bS));
          mbar_arrive(bar(bVEmpty + (it & 1)));
        }
      }
      if (!ok) break;
      if (j.chunks > 0) {
        ok = wait_warp(bKV, (uint32_t)it - 1);
        if (!ok) break;
        tc_fence_after();
      }
      if (j.fin) {
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {
          float s[32];
          if (j.chunks > 0) {
            tmem_ld32(row + 32 * p, s);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float4 y = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
            if (j.chunks == 0)
              y = init ? *reinterpret_cast<const float4*>(init + 32 * p + i)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(j.fin + dv * D + 32 * p + i) = y;
          }
        }
      }
      if (j.decay && dv == 0) *j.decay = exp2_approx(decay);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------- segments
// With few chains a sequence is cut into segments of `L` chunks that run at once: a first
// pass forms every segment's end state from a zero state (the first from h0), a scan turns
// them into the states entering the segments,
//     S_in(0) = h0,   S_in(1) = S_end(0),   S_in(k+1) = S_end(k) + (segment k's decay) S_in(k),
// and the pass with outputs starts each segment from its own (also the first, so that hT
// may be h0: h0 is not read any more when a last segment writes hT).
__global__ void __launch_bounds__(1024) lin_seg_plan_kernel(LinArgs a, int L, int4* tab,
                                                            int* first, int* n_segs, int cap) {
  __shared__ int warp_sums[32];
  __shared__ int carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int b = 0; b < a.n_seqs; b += blockDim.x) {
    const int n = b + tid;
    int64_t t0 = 0, t1 = 0;
    int P = 0;
    if (n < a.n_seqs) {
      seq_range(a, n, t0, t1);
      const int64_t per = (int64_t)L * C;
      P = t1 > t0 ? (int)((t1 - t0 + per - 1) / per) : 1;
    }
    int v = P;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int w = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sums[lane] = w;
    }
    __syncthreads();
    const int f = carry + v - P + (warp > 0 ? warp_sums[warp - 1] : 0);
    if (n < a.n_seqs) {
      first[n] = min(f, cap);
      for (int k = 0; k < P && f + k < cap; ++k) {
        const int64_t s0 = t0 + (int64_t)k * L * C;
        const int64_t s1 = min(t1, s0 + (int64_t)L * C);
        tab[f + k] = make_int4(n, (int)s0, (int)(s1 - s0), k | (k == P - 1 ? (int)0x80000000 : 0));
      }
    }
    __syncthreads();
    if (tid == (int)blockDim.x - 1) carry = f + P;
    __syncthreads();
  }
  if (tid == 0) {
    first[a.n_seqs] = min(carry, cap);
    *n_segs = min(carry, cap);
  }
}

constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) lin_seg_scan_kernel(
    const int* __restrict__ first, int H, const float* __restrict__ h0,
    const float* __restrict__ s_end,
    const float* __restrict__ decay, float* __restrict__ s_in) {
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit - (int64_t)n * H);
  const int64_t e = 4 * ((int64_t)blockIdx.y * kScanThreads + threadIdx.x);
  const int f0 = __ldg(first + n), f1 = __ldg(first + n + 1);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h0) s = *reinterpret_cast<const float4*>(h0 + unit * D * D + e);
  if (f0 < f1) *reinterpret_cast<float4*>(s_in + ((int64_t)f0 * H + h) * D * D + e) = s;
  for (int f = f0; f + 1 < f1; ++f) {
    const int64_t at = ((int64_t)f * H + h) * D * D + e;
    const float4 x = *reinterpret_cast<const float4*>(s_end + at);
    const float d = f == f0 ? 0.f : __ldg(decay + (int64_t)f * H + h);
    s = f == f0 ? x : make_float4(fmaf(d, s.x, x.x), fmaf(d, s.y, x.y), fmaf(d, s.z, x.z),
                                  fmaf(d, s.w, x.w));
    *reinterpret_cast<float4*>(s_in + at + (int64_t)H * D * D) = s;
  }
}

struct SegLayout {
  int4* tab;
  int *first, *n_segs;
  float *decay, *s_end, *s_in;
  int cap;
  size_t bytes;
};

SegLayout seg_layout(void* ws, int64_t n_tokens, int n_seqs, int H, int L) {
  SegLayout l{};
  uint8_t* base = static_cast<uint8_t*>(ws);
  size_t off = 0;
  auto take = [&](size_t b) {
    uint8_t* p = base + off;
    off += (b + 255) & ~size_t(255);
    return p;
  };
  l.cap = (int)(n_tokens / ((int64_t)L * C) + n_seqs);
  l.n_segs = reinterpret_cast<int*>(take(sizeof(int)));
  l.first = reinterpret_cast<int*>(take(sizeof(int) * ((size_t)n_seqs + 1)));
  l.tab = reinterpret_cast<int4*>(take(sizeof(int4) * (size_t)l.cap));
  const size_t units = (size_t)l.cap * H;
  l.decay = reinterpret_cast<float*>(take(sizeof(float) * units));
  l.s_end = reinterpret_cast<float*>(take(sizeof(float) * units * D * D));
  l.s_in = reinterpret_cast<float*>(take(sizeof(float) * units * D * D));
  l.bytes = off;
  return l;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 128 tokens x 64 channels of one head of a [tokens][heads][128] bf16 tensor.
cudaError_t encode_tiles(CUtensorMap* map, const void* p, int heads, int64_t n_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
  const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)C};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool kOut>
cudaError_t run(const CUtensorMap* tm, const LinArgs& a, int64_t items, const char* name,
                cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      lin_tc_kernel<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  ProfScope prof_scope(name, s);
  lin_tc_kernel<kOut><<<(unsigned)(items < sms ? items : sms), kThreads, kSmemBytes, s>>>(
      tm[0], tm[1], tm[2], a);
  return cudaGetLastError();
}

}  // namespace

// Chunks of a segment, 0: sequences are not cut.
int linear_segment_chunks(int64_t n_tokens, int n_seqs, int H, int forced, bool sequential) {
  if (sequential || n_tokens == 0) return 0;
  if (forced > 0) return forced;
  const int64_t sms = sm_count(), chains = (int64_t)n_seqs * H;
  const int64_t chunks = (n_tokens / C + n_seqs) / n_seqs;  // of an average sequence
  if (2 * chains > sms || chunks < 16) return 0;
  int64_t P = sms / chains;
  if (P > chunks / 4) P = chunks / 4;
  return (int)((chunks + P - 1) / P);
}

size_t linear_tc_workspace_bytes(int64_t n_tokens, int n_seqs, int H, int seg_chunks) {
  return seg_chunks > 0 ? seg_layout(nullptr, n_tokens, n_seqs, H, seg_chunks).bytes : 256;
}

cudaError_t launch_linear_tc(const void* q, const void* k, const void* v, const float* g,
                             int g_head, float scale, const float* h0, const int32_t* cu,
                             int64_t T_per_seq, void* o, float* hT, int64_t n_tokens, int n_seqs,
                             int H, int Hk, int seg_chunks, void* ws, int* err, cudaStream_t s) {
  LinArgs a{};
  a.g = g;
  a.g_head = g_head;
  a.scale = scale;
  a.h0 = h0;
  a.cu = cu;
  a.T = T_per_seq;
  a.n_tokens = n_tokens;
  a.n_seqs = n_seqs;
  a.H = H;
  a.rep = H / Hk;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.hT = hT;
  a.err = err;
  CUtensorMap tm[3];
  memset(tm, 0, sizeof(tm));
  cudaError_t e = cudaSuccess;
  if (n_tokens > 0) {  // with no tokens there are no chunks to copy
    e = encode_tiles(&tm[0], q, Hk, n_tokens);
    if (e == cudaSuccess) e = encode_tiles(&tm[1], k, Hk, n_tokens);
    if (e == cudaSuccess) e = encode_tiles(&tm[2], v, H, n_tokens);
    if (e != cudaSuccess) return e;
  }
  if (seg_chunks <= 0) return run<true>(tm, a, (int64_t)n_seqs * H, "kda_linear_tc", s);
  const SegLayout l = seg_layout(ws, n_tokens, n_seqs, H, seg_chunks);
  {
    ProfScope prof_scope("kda_linear_seg_plan", s);
    lin_seg_plan_kernel<<<1, 1024, 0, s>>>(a, seg_chunks, l.tab, l.first, l.n_segs, l.cap);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  a.tab = l.tab;
  a.n_segs = l.n_segs;
  a.s_in = l.s_in;
  a.s_end = l.s_end;
  a.seg_decay = l.decay;
  e = run<false>(tm, a, (int64_t)l.cap * H, "kda_linear_tc_state", s);
  if (e != cudaSuccess) return e;
  {
    ProfScope prof_scope("kda_linear_seg_scan", s);
    lin_seg_scan_kernel<<<dim3((unsigned)((int64_t)n_seqs * H), D * D / 4 / kScanThreads),
                          kScanThreads, 0, s>>>(l.first, H, h0, l.s_end, l.decay, l.s_in);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return run<true>(tm, a, (int64_t)l.cap * H, "kda_linear_tc", s);
}

}  // namespace kda
