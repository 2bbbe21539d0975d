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
//     QS   O = Q S, from a bf16 copy of S^T    (lanes = tokens); then O_i *= scale e^{G_i}
//     KV   S^T += Vw^T K, Vw_j = e^{G_C - G_j} v_j, after S^T *= e^{G_C}
//     PV   O += P V with P = scale * decay * scores, bf16
// Rounding: P and the copy of S to bf16 (o is bf16 as well, each adds an error of the size
// of o's own rounding).  The final state is fp32, so Vw is kept as two bf16 parts, hi + lo
// (16 bits of each weighted value: off by 2^-14.9 at most and 4.4e-6 rms, so hT is off by 4.2e-6
// where fp32 sums are by 2e-7), and KV is issued for both.  A third part costs more than it gives:
// tensor memory has no room for it but the outputs' columns, which makes the weighted values wait
// for the last chunk's outputs (8192 tokens x 96 heads, when it was tried, 173 -> 244 us for 18
// bits, 268 with an fp32 split for all 24).
//
// What bounds a chunk is shared-memory bandwidth (128 bytes a clock): an M = N = 128 MMA
// reads 128 bytes of operands a clock when both come from shared memory.  So P and both
// parts of Vw are A operands in tensor memory, k and v tiles are used as the tensor copies
// left them (128-byte swizzled: the same bytes are a K-major operand where channels are
// contracted and an MN-major one where tokens are), and v reaches the lanes of its channels
// by transposing matrix loads.  What is left a chunk: 224 KB of MMA operands, 96 KB of
// copies, about as much again by the groups below, of 5300 clocks (678 KB) that a chunk takes
// at one chain an SM; at all SMs busy a chunk takes 5800 and HBM bounds it.  Measured: 8192
// tokens x 96 heads (96 of 152 SMs have a chain) 178 us, 4.6 TB/s; 14 ragged sequences of 17589
// tokens x 48 heads 183 us, 5.2 TB/s; 131072 tokens x 16 heads in segments 498 to 520 us.  Handing
// chains out as jobs of a warp of their own, by ticket where there are several a CTA, cost the
// first case 174 -> 178 us and brought the second from 235 to 199.
//
// The ring holds two whole chunks of q, k and v.
//
// Warps: copies, MMA issue, decay records, jobs; then six groups of four, one warp of each on
// every SM sub-partition: weighted values, scores -> P (two, half the keys each), outputs
// (two, half the channels each), state.  The record warp hands every chunk to the others as
// one record in shared memory.  Loops stay rolled and jobs are decoded once: eight roles run
// at the same time, and with 94 KB of code instruction fetch bounded the kernel (8500 clocks
// a chunk).
//
// Decays.  With L_i the sum of g inside a 32-token block up to i, U_j the sum behind j in
// its block and T_b the block totals, every exponent but those inside a diagonal block is
// a sum of non-positive terms: e^{G_i - G_j} = e^{L_i + T between} e^{U_j}, so a decay is
// as exact as fp32 addition next to any g.  Inside a block it is e^{L_i - L_j}, two sums that
// start at the block: behind several g of -100 in it the difference keeps about 3e-4, next to the
// rounding of P (2^-8).  g is held at -100 at least (e^-100 is 0 in fp32), which also makes -inf
// drop the state.
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

constexpr uint32_t kTileBytes = C * D * 2;  // 32 KB: two 64-channel blocks of 128 rows
constexpr uint32_t kHalfTile = kTileBytes / 2;
enum { tK = 0, tV = 1, tQ = 2 };            // tile t of chunk `it` sits in slot 3 (it & 1) + t
constexpr uint32_t kSbOff = 6 * kTileBytes;  // bf16 copy of S^T, K-major
constexpr uint32_t kVecOff = kSbOff + kTileBytes;

// A chunk as the record warp hands it out: what it is, and its decays (log2 units).
struct __align__(16) Rec {
  float L[C];    // sum of g inside the token's 32-token block, inclusive
  float cf[C];   // 2^(sum of g behind the token inside its block)
  float T[4];    // block totals
  float aft[4];  // 2^(totals of the blocks behind)
  const float* init;  // first chunk of a job: state to start from (null: zero)
  float* fin;         // last chunk of a job: where the state goes (null: nowhere)
  float* decay;       // last chunk: where the job's whole decay goes (null: nowhere)
  int tok, len, h, flags;
  float total;   // of the chunk
  float sofar;   // of the job, with this chunk
};
enum { kFirst = 1, kLast = 2, kStop = 4 };
// A chain (or a segment of one), as the scheduling warp hands it out.
struct Job {
  const float* init;
  float* fin;
  float* decay;
  int tok, tokens, h, stop;
};
constexpr uint32_t kJobOff = kVecOff + 2 * sizeof(Rec);
constexpr uint32_t kBarOff = kJobOff + 2 * sizeof(Job);
constexpr uint32_t kBarBytes = 32 * 8;
constexpr uint32_t kSmemUsed = kBarOff + kBarBytes + 16;
constexpr uint32_t kSmemBytes = 232448;  // all an SM has: one CTA each
static_assert(kSmemUsed <= kSmemBytes, "shared memory");

// barriers
enum {
  bFull = 0,           // [6] tile landed
  bEmpty = bFull + 6,  // [6] tile free again
  bRFull = bEmpty + 6,  // [2] record written
  bREmpty = bRFull + 2,  // [2] record read
  bJFull = bREmpty + 2,  // [2] job written
  bJNext = bJFull + 2,   // the next job is wanted and has room
  bQK = bJNext + 1,    // scores complete
  bVw = bQK + 1,       // [2] weighted values of tokens 0-63, 64-127 written
  bP = bVw + 2,        // P written
  bS = bP + 1,         // state scaled and copied
  bKV = bS + 1,        // state updated
  bQS = bKV + 1,       // Q S complete
  bOs = bQS + 1,       // O scaled
  bPV = bOs + 1,       // outputs complete
  bO = bPV + 1,        // outputs read out
  bZ = bO + 1,         // rows past a sequence's end cleared
  bDrain = bZ + 1,
  kBars = bDrain + 1
};
static_assert(kBars * 8 <= kBarBytes, "barriers");

// TMEM columns: state, scores (P over the left half of each half of them), O, weighted values hi and lo
constexpr uint32_t kT_S = 0, kT_P = 128, kT_O = 256, kT_Vhi = 384, kT_Vlo = 448;

constexpr int kGroup = 128;
constexpr int kThreads = 128 + 6 * kGroup;  // scores and outputs take two groups each
// A wait gives up after this many polls.  A poll that nothing ends was measured to take 3.8 us
// (at this hint of 1 us), so a wait ends after 16 s; the longest that is meant to be waited for is
// a chain's end, 2.4 us a chunk: 8e8 tokens of one head, more than the memory holds.
constexpr uint32_t kPolls = 1u << 22, kPollNs = 1000;

// Waits for the phase of `parity` to complete; 0 if it has not after kPolls polls.  (The loop
// is all there is to a wait site: a role whose wait fails reports that where it ends.)
__device__ __forceinline__ uint32_t wait_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n\t"
      "POLL:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra POLL;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity & 1u), "n"(kPolls), "n"(kPollNs)
      : "memory");
  return ok;
}

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
  int* ticket;          // next job (null: every gridDim.x-th, from blockIdx.x)
  const int* order;     // sequences by falling length (null: as they come)
  int* err;
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
  if (bad) atomicExch(a.err, kDevErrBadSeqlens);
}

template <bool kOut>
__device__ __forceinline__ int job_count(const LinArgs& a) {
  return (a.tab ? *a.n_segs : a.n_seqs) * a.H;
}

template <bool kOut>
__device__ __forceinline__ Job get_job(const LinArgs& a, int item) {
  Job j{};
  int u = item / a.H;
  j.h = item - u * a.H;
  if (a.order) {
    u = a.order[u];
    item = u * a.H + j.h;
  }
  if (!a.tab) {
    int64_t t0, t1;
    seq_range(a, u, t0, t1);
    j.tok = (int)t0;
    j.tokens = (int)(t1 - t0);
    const int64_t s = (int64_t)item * D * D;
    j.init = a.h0 ? a.h0 + s : nullptr;
    j.fin = a.hT ? a.hT + s : nullptr;
  } else {
    const int4 e = a.tab[u];
    j.tok = e.y;
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
  return j;
}

// The issuing warps run their control flow with all lanes, so that descriptors, addresses
// and loop counters stay in the warp's uniform registers, where these instructions take
// them from; `lead` (1 on one lane) predicates the instruction alone.  (Issued from inside
// a one-lane branch every operand was moved over first: 110 to 250 clocks an MMA that the
// tensor pipe finishes in 64.)
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t ad, uint64_t bd,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t at, uint64_t bd,
                                       uint32_t idesc) {  // accumulates
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Both 64-channel boxes of a tile, completing on `bar`.
__device__ __forceinline__ void load_tile(uint32_t lead, uint32_t dst, const void* tmap, int head,
                                          int tok, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 st;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%5], %7;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%2, {0, %3, %4}], [%5];\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%1], [%2, {64, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "r"(dst + kHalfTile), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(head), "r"(tok), "r"(bar),
      "r"(lead), "r"(kTileBytes)
      : "memory");
}

// Four transposed 8 x 8 bf16 matrices; lane l gives the address of row l % 8 of matrix l / 8
// and gets, of each, column l / 4 of rows 2 (l % 4) and + 1 as one pair.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes x 32 columns: of each four columns, registers 2i and 2i + 1 of lane l go to TMEM
// lanes l / 4 and l / 4 + 8, column 4 i + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// v (wh + wl) of a bf16 pair in two bf16 parts: hi = v wh rounded; v wh - hi has at most
// eight significant bits and is exact; v wl joins it with the second rounding.
__device__ __forceinline__ void weigh(uint32_t v, uint32_t wh, uint32_t wl, uint32_t& hi,
                                      uint32_t& lo) {
  asm("{\n\t.reg .b32 n, r, z;\n\t"
      "mov.b32 z, 0x80008000;\n\t"  // -0: the product alone, its sign kept
      "fma.rn.bf16x2 %0, %2, %3, z;\n\t"
      "neg.bf16x2 n, %0;\n\t"
      "fma.rn.bf16x2 r, %2, %3, n;\n\t"
      "fma.rn.bf16x2 %1, %2, %4, r;\n\t}"
      : "=&r"(hi), "=&r"(lo)
      : "r"(v), "r"(wh), "r"(wl));
}
// 16 lanes x 64 columns: registers 4 i + 2 r + e of lane l hold TMEM lane l / 4 + 8 r, column
// 8 i + 2 (l % 4) + e.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Within each four lanes: word j of lane q becomes word q of lane j.
__device__ __forceinline__ void transpose4(uint32_t (&z)[4], int lane) {
#pragma unroll
  for (int m = 2; m >= 1; m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & m) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? z[k] : z[k + m], m);
      if (up) z[k] = got;
      else z[k + m] = got;
    }
  }
}

// kOut: outputs and final states.  Otherwise the state alone (the first pass over segments).
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    lin_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const LinArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  if (pad + kSmemUsed > kSmemBytes) {  // (uniform; dynamic shared memory starts aligned)
    if (threadIdx.x == 0) atomicExch(a.err, kDevErrTimeout);
    return;
  }
  uint8_t* sm = smem_raw + pad;
  const uint32_t base = smem_addr(sm);
  const uint32_t bars = base + kBarOff;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBarOff + kBarBytes);
  Rec* recs = reinterpret_cast<Rec*>(sm + kVecOff);
  Job* jobs = reinterpret_cast<Job*>(sm + kJobOff);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  bool done = false;  // this role has come to the end of the work

  if (t == 0) {
    // arrivals a phase: copies, commits and single threads 1, groups one a warp, records one
    // a warp that reads them
    constexpr uint32_t k4 = 3u << bVw | 1u << bS | 1u << bZ;
    constexpr uint32_t k8 = 1u << bP | 1u << bOs | 1u << bO;
    constexpr uint32_t kRec = 3u << bREmpty;
#pragma unroll 1
    for (int i = 0; i < kBars; ++i) {
      const uint32_t b = 1u << i;
      const int n = b & kRec ? (kOut ? 25 : 9) : (b & k8 ? 8 : (b & k4 ? 4 : (i == bJNext ? 2 : 1)));
      mbar_init(bar(i), (uint32_t)n);
    }
    mbar_fence_init();
  }
  if (warp == 3) tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  wait_previous();
  release_next();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](int b, uint32_t parity) { return wait_poll(bar(b), parity) != 0; };
  // the same for a whole warp: one outcome, so that warp-wide instructions stay together
  auto wait_warp = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(b, parity)) != 0;
  };
  auto arrive = [&](int b) {  // once a warp, after all of its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  auto full = [](int tile, int it) { return bFull + 3 * (it & 1) + tile; };
  auto empty = [](int tile, int it) { return bEmpty + 3 * (it & 1) + tile; };
  auto slot = [](int tile, int it) { return (uint32_t)(3 * (it & 1) + tile) * kTileBytes; };

  if (warp == 0) {
    // ------------------------------------------------------------------ copies in
    constexpr int kTiles = kOut ? 3 : 2;
    const uint32_t lead = elect_lane();
    auto tile_at = [](int x) { return x == 0 ? tK : (kOut && x == 1 ? tQ : tV); };
    int it = 0, m = 0;  // chunks, tiles copied
    bool ok = true;
#pragma unroll 1
    for (int n = 0;; ++n) {
      ok = wait_warp(bJFull + (n & 1), (uint32_t)(n >> 1));
      if (!ok) break;
      const Job j = jobs[n & 1];
      if (j.stop) break;
      const int kv_head = j.h / a.rep;
      // the next job is asked for two chunks before this one's end: late, so that CTAs that
      // draw jobs by ticket end together, and early enough for its decoding
      const int ask = j.tokens - 2 * C;
      if (ask <= 0) arrive(bJNext);
#pragma unroll 1
      for (int c = 0; c < j.tokens && ok; c += C, ++it) {
        if (c < ask && c + C >= ask) arrive(bJNext);
#pragma unroll 1
        for (int x = 0; x < kTiles; ++x) {  // in the order their slots fall free
          const int i = tile_at(x);
          ok = it < 2 || wait_warp(empty(i, it), (uint32_t)(it >> 1) - 1);
          if (!ok) break;
          const void* tm = i == tK ? &tm_k : (i == tQ ? &tm_q : &tm_v);
          load_tile(lead, base + slot(i, it), tm, i == tV ? j.h : kv_head, j.tok + c,
                    bar(full(i, it)));
          ++m;
        }
      }
      if (!ok) break;
    }
    done = ok;
    if (!ok) {  // copies in flight must land before the CTA exits
#pragma unroll 1
      for (int x = max(0, m - 2 * kTiles); x < m; ++x)
        wait(full(tile_at(x % kTiles), x / kTiles), (uint32_t)(x / kTiles >> 1));
    }
  } else if (warp == 2) {
    // --------------------------------------------------------------------- records
    // One a chunk (a job without tokens is one record, the end of the work another); the
    // next chunk's g is on its way while this one's sums are formed.
    int d = 0, n = 0, c = 0;
    float gn[4];
    float sofar = 0.f;
    Job j;
    bool ok = true;
    auto next_job = [&]() {
      ok = wait_warp(bJFull + (n & 1), (uint32_t)(n >> 1));
      j = jobs[n & 1];
      arrive(bJNext);  // (the job before this one needs its place no more)
      ++n;
    };
    auto fetch = [&]() {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int r = c + 32 * b + lane;
        gn[b] = 0.f;
        if (ok && r < j.tokens)
          gn[b] = __ldg(a.g + (a.g_head ? (int64_t)j.h : (int64_t)(j.tok + r) * a.H + j.h));
      }
    };
    next_job();
    fetch();
#pragma unroll 1
    for (; ok; ++d) {
      // this record's job and g; then on to the next chunk or job, whose g is fetched here
      const Job jc = j;
      const int cc = c;
      const bool last = cc + C >= jc.tokens, end = jc.stop != 0;
      float g[4], u[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) g[b] = gn[b];
      if (!end) {
        c += C;
        if (last) {
          c = 0;
          next_job();
          if (!ok) break;
        }
        fetch();
      }
      ok = d < 2 || wait_warp(bREmpty + (d & 1), (uint32_t)(d >> 1) - 1);
      if (!ok) break;
      Rec& v = recs[d & 1];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        g[b] = (g[b] < kMinG ? kMinG : g[b]) * kLog2e;  // NaN stays NaN
        u[b] = __shfl_down_sync(0xffffffffu, g[b], 1);
        if (lane == 31) u[b] = 0.f;
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float x = __shfl_up_sync(0xffffffffu, g[b], o);
          const float y = __shfl_down_sync(0xffffffffu, u[b], o);
          if (lane >= o) g[b] += x;
          if (lane + o < 32) u[b] += y;
        }
      float after = 0.f;
#pragma unroll
      for (int b = 3; b >= 0; --b) {
        v.L[32 * b + lane] = g[b];
        v.cf[32 * b + lane] = exp2_approx(u[b]);
        const float T = __shfl_sync(0xffffffffu, g[b], 31);
        if (lane == 0) {
          v.T[b] = T;
          v.aft[b] = exp2_approx(after);
        }
        after += T;
      }
      sofar = cc == 0 ? after : sofar + after;
      if (lane == 0) {
        v.init = jc.init;
        v.fin = jc.fin;
        v.decay = jc.decay;
        v.tok = jc.tok + cc;
        v.len = min(C, jc.tokens - cc);
        v.h = jc.h;
        v.flags = end ? kStop : ((cc == 0 ? kFirst : 0) | (last ? kLast : 0));
        v.total = after;
        v.sofar = sofar;
      }
      arrive(bRFull + (d & 1));
      if (end) break;
    }
    done = ok;
  } else if (warp == 1) {
    // -------------------------------------------------------------------- MMAs
    // Order a chunk: KV, QS, PV, then QK of the next chunk.  KV comes first: the state group
    // works on its result, the next chunk's first operand, while the others run.
    const uint32_t lead = elect_lane();
    const uint32_t id_kk = idesc_bf16_mn(C, C, 0, 0);  // both operands K-major
    const uint32_t id_kn = idesc_bf16_mn(C, D, 0, 1);  // B MN-major
    bool ok = true, any = false;
    int d = 0;
    // D = A B^T over 128 channels, both tiles K-major
    auto mma_kk = [&](uint32_t dst, uint32_t at, uint32_t bt) {
      const uint64_t da = kmajor_desc(at, C, 0), db = kmajor_desc(bt, C, 0);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint32_t off = (uint32_t)(s >> 2) * kHalfTile + (uint32_t)(s & 3) * 32u;
        mma_ss(lead, dst, desc_advance(da, off), desc_advance(db, off), id_kk, s > 0);
      }
    };
#pragma unroll 1
    for (int it = -1; ok; ++it) {
      const uint32_t par = (uint32_t)it;
      if (it >= 0) {
        ok = wait_warp(bS, par);
        if (!ok) break;
        tc_fence_after();
        ok = kOut || wait_warp(full(tK, it), par >> 1);  // (with outputs QK has waited for k)
        if (!ok) break;
        any = true;
        uint64_t dk = mnmajor_desc_lbo(base + slot(tK, it), kHalfTile, 1024, 0);
        uint32_t va = tmem + kT_Vhi;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {  // tokens 0-63, 64-127
          ok = wait_warp(bVw + hf, par);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint64_t b = desc_advance(dk, (uint32_t)s * 2048u);
            mma_ts(lead, tmem + kT_S, va + (kT_Vlo - kT_Vhi) + 8 * s, b, id_kn);
            mma_ts(lead, tmem + kT_S, va + 8 * s, b, id_kn);
          }
          dk = desc_advance(dk, 4 * 2048);
          va += 32;
        }
        if (!ok) break;
        commit_to(lead, bar(bKV));
        commit_to(lead, bar(empty(tK, it)));
        if (kOut) {
          ok = it == 0 || wait_warp(bO, par - 1);
          if (!ok) break;
          tc_fence_after();
          mma_kk(tmem + kT_O, base + slot(tQ, it), base + kSbOff);
          commit_to(lead, bar(bQS));
          commit_to(lead, bar(empty(tQ, it)));
          ok = wait_warp(bP, par) && wait_warp(bOs, par);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = mnmajor_desc_lbo(base + slot(tV, it), kHalfTile, 1024, 0);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_ts(lead, tmem + kT_O, tmem + kT_P + (uint32_t)(8 * s + (s & 4) * 8), desc_advance(dv, (uint32_t)s * 2048u),
                   id_kn);
          commit_to(lead, bar(bPV));
        }
        commit_to(lead, bar(empty(tV, it)));
      }
      int len = 0;  // the next record that is a chunk
#pragma unroll 1
      while (len <= 0) {
        ok = wait_warp(bRFull + (d & 1), (uint32_t)(d >> 1));
        if (!ok) break;
        len = recs[d & 1].len;
        const int flags = recs[d & 1].flags;
        arrive(bREmpty + (d & 1));
        ++d;
        done = __any_sync(0xffffffffu, (flags & kStop) != 0) != 0;
        ok = !done;
        if (!ok) break;
        len = __shfl_sync(0xffffffffu, len, 0);
      }
      if (!ok) break;
      if (kOut) {
        const uint32_t ph = (uint32_t)((it + 1) >> 1);
        ok = wait_warp(full(tK, it + 1), ph) && wait_warp(full(tQ, it + 1), ph);
        if (!ok) break;
        tc_fence_after();
        mma_kk(tmem + kT_P, base + slot(tQ, it + 1), base + slot(tK, it + 1));
        commit_to(lead, bar(bQK));
        any = true;
      }
    }
    if (!done && any) {  // drain MMAs in flight
      commit_to(lead, bar(bDrain));
      wait(bDrain, 0);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------------ jobs
    const int items = job_count<kOut>(a);
    int item = blockIdx.x;
#pragma unroll 1
    for (int n = 0;; ++n) {
      Job j{};
      j.stop = item >= items;
      if (!j.stop) j = get_job<kOut>(a, item);
      if (lane == 0) jobs[n & 1] = j;
      arrive(bJFull + (n & 1));
      done = j.stop != 0;
      if (done || !wait_warp(bJNext, (uint32_t)n)) break;
      if (a.ticket) {
        if (lane == 0) item = (int)gridDim.x + atomicAdd(a.ticket, 1);
        item = __shfl_sync(0xffffffffu, item, 0);
      } else {
        item += (int)gridDim.x;
      }
    }
  } else if (warp >= 4) {
    // The four groups: records in order, each with its own work on a chunk.
    const int group = (warp >> 2) - 1, w = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    const int row = 32 * w + lane;
    if (group == 0) {
      // -------------------------------------------------------- weighted values
      // Warp w takes value rows 32 w .. + 31: a transposing load brings 16 rows x 16
      // tokens, a lane holding token pairs of one row, as the 16-lane stores to tensor
      // memory want them.  Rows of k and v past the sequence's end hold other tokens: the
      // group clears them first, so that nothing of them (a NaN) meets this sequence.
      // matrix m of a load: value rows 8 (m & 1), tokens 8 (m >> 1); this lane's row of it
      const int mrow = (lane & 7) + 8 * (lane >> 4), mdv = (lane >> 3) & 1;
      int it = 0, cleared = 0;
#pragma unroll 1
      for (int d = 0;; ++d) {
        if (!wait_warp(bRFull + (d & 1), (uint32_t)(d >> 1))) break;
        const Rec& v = recs[d & 1];
        const int len = v.len, flags = v.flags;
        done = (flags & kStop) != 0;
        if (done) break;
        if (len > 0) {
          const uint32_t ph = (uint32_t)(it >> 1);
          bool ok = wait_warp(full(tV, it), ph) &&
                    (it == 0 || wait_warp(bKV, (uint32_t)it - 1));  // the last chunk's are read
          if (ok && len < C) {
            ok = wait_warp(full(tK, it), ph) && (!kOut || wait_warp(bQK, (uint32_t)it));
            if (!ok) break;
#pragma unroll 1
            for (int e = row; e < (C - len) * 16; e += kGroup) {
              const uint32_t off = (uint32_t)((e >> 3) & 1) * kHalfTile +
                                   (uint32_t)((len + (e >> 4)) * 128 + (e & 7) * 16);
              *reinterpret_cast<uint4*>(sm + slot(tV, it) + off) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(sm + slot(tK, it) + off) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            arrive(bZ);
            ok = wait_warp(bZ, (uint32_t)cleared++);
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t vt = base + slot(tV, it) + (uint32_t)(w >> 1) * kHalfTile;
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {  // tokens 64 hf .. + 63
            // weights of this lane's token pairs, eight tokens apart, in two bf16 parts
            uint32_t wh[8], wl[8];
            const int pt = 64 * hf + 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float f = v.aft[2 * hf + (i >> 2)];
              const float2 c = __fmul2_rn(*reinterpret_cast<const float2*>(&v.cf[pt + 8 * i]),
                                          make_float2(f, f));
              wh[i] = pack_bf16(c.x, c.y);
              wl[i] = pack_bf16(c.x - bf16_lo(wh[i]), c.y - bf16_hi(wh[i]));
            }
#pragma unroll 1
            for (int dh = 0; dh < 2; ++dh) {  // 16 value rows
              uint32_t hi[16], lo[16];
              const uint32_t src = vt + (uint32_t)((64 * hf + mrow) * 128 +
                                                   (((4 * (w & 1) + 2 * dh + mdv) ^ (lane & 7)) << 4));
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // 16 tokens
                uint32_t y[4];
                ldmatrix4_trans(src + 2048u * i, y);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                  weigh(y[m], wh[2 * i + (m >> 1)], wl[2 * i + (m >> 1)], hi[4 * i + m], lo[4 * i + m]);
              }
              const uint32_t dst = lanes + ((uint32_t)(16 * dh) << 16) + 32u * hf;
              tmem_st_16x128b_x8(dst + kT_Vhi, hi);
              tmem_st_16x128b_x8(dst + kT_Vlo, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(bVw + hf);
          }
          ++it;
        }
        arrive(bREmpty + (d & 1));
      }
    } else if (group <= 2) {
      if constexpr (kOut) {
      // ------------------------------------------------------------ scores -> P
      // Two groups, thread = token row and 64 of its keys, 32 at a time.  P (packed pairs)
      // overwrites the left half of the group's own scores, behind the scores being read.
      const int b0 = 2 * (group - 1);  // first of the group's two key blocks
      const uint32_t col = lanes + kT_P;
      int it = 0;
#pragma unroll 1
      for (int d = 0;; ++d) {
        if (!wait_warp(bRFull + (d & 1), (uint32_t)(d >> 1))) break;
        const Rec& v = recs[d & 1];
        const int len = v.len, flags = v.flags;
        done = (flags & kStop) != 0;
        if (done) break;
        if (len > 0) {
          if (!wait_warp(bQK, (uint32_t)it)) break;
          tc_fence_after();
          const float Li = v.L[row];
#pragma unroll 1
          for (int b = b0; b < b0 + 2; ++b) {
            float s[32];
            uint32_t pk[16];
            if (b > w) {  // keys behind every token of this warp
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            } else {
              tmem_ld32(col + 32 * b, s);
              float upto = Li;  // decay exponent from the end of the key block to this token
#pragma unroll
              for (int x = 1; x < 3; ++x) upto += (x > b && x < w) ? v.T[x] : 0.f;
              const float r = a.scale * exp2_approx(upto);
              const float2 r2 = make_float2(r, r);
              tmem_wait_ld();
              if (b < w) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 f = *reinterpret_cast<const float4*>(&v.cf[32 * b + i]);
                  const float2 p = __fmul2_rn(__fmul2_rn(make_float2(f.x, f.y), r2),
                                              make_float2(s[i], s[i + 1]));
                  const float2 q = __fmul2_rn(__fmul2_rn(make_float2(f.z, f.w), r2),
                                              make_float2(s[i + 2], s[i + 3]));
                  pk[i / 2] = pack_bf16(p.x, p.y);
                  pk[i / 2 + 1] = pack_bf16(q.x, q.y);
                }
              } else {  // the diagonal block
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
            tmem_st16(col + 32 * b0 + 16 * (b - b0), pk);
          }
          tmem_wait_st();
          tc_fence_before();
          arrive(bP);
          ++it;
        }
        arrive(bREmpty + (d & 1));
      }
      } else {
        done = true;
      }
    } else if (group <= 4) {
      if constexpr (kOut) {
      // --------------------------------------------------------------- outputs
      // Two groups, thread = token row and 64 of its channels: O *= scale e^{G_i} between QS and
      // PV; then the rows that the sequence has go from the registers to memory.
      const int half = group - 3;
      const uint32_t col = lanes + kT_O + 64 * half;
      int it = 0;
#pragma unroll 1
      for (int d = 0;; ++d) {
        if (!wait_warp(bRFull + (d & 1), (uint32_t)(d >> 1))) break;
        const Rec& v = recs[d & 1];
        const int len = v.len, flags = v.flags, h = v.h, tok = v.tok;
        float e0 = v.L[row];
#pragma unroll
        for (int b = 0; b < 3; ++b) e0 += b < w ? v.T[b] : 0.f;
        arrive(bREmpty + (d & 1));
        done = (flags & kStop) != 0;
        if (done) break;
        if (len <= 0) continue;
        const float e1 = a.scale * exp2_approx(e0);
        const float2 e2 = make_float2(e1, e1);
        if (!wait_warp(bQS, (uint32_t)it)) break;
        tc_fence_after();
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          float y[32];
          tmem_ld32(col + 32 * p, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 z = __fmul2_rn(make_float2(y[i], y[i + 1]), e2);
            y[i] = z.x;
            y[i + 1] = z.y;
          }
          tmem_st32(col + 32 * p, y);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bOs);
        if (!wait_warp(bPV, (uint32_t)it)) break;
        tc_fence_after();
        // 16 rows x 64 channels at a time, four lanes a row; lane q of them holds pairs
        // 8 i + 2 q, and a 4 x 4 exchange of pairs leaves it channels 8 q .. 8 q + 7
        __nv_bfloat16* orow = a.o + ((int64_t)(tok + 32 * w + (lane >> 2)) * a.H + h) * D + 64 * half +
                              8 * (lane & 3);
#pragma unroll 1
        for (int sl = 0; sl < 2; ++sl) {
          uint32_t y[32];
          tmem_ld_16x256b_x8(col + ((uint32_t)(16 * sl) << 16), y);
          tmem_wait_ld();
          if (sl == 1) {
            tc_fence_before();
            arrive(bO);
          }
#pragma unroll
          for (int rs = 0; rs < 2; ++rs) {  // rows 0-7, 8-15 of them
            const int r = 16 * sl + 8 * rs;
            const bool in = 32 * w + (lane >> 2) + r < len;
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // channels 32 g .. + 31
              uint32_t z[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                z[i] = pack_bf16(__uint_as_float(y[4 * (4 * g + i) + 2 * rs]),
                                 __uint_as_float(y[4 * (4 * g + i) + 2 * rs + 1]));
              transpose4(z, lane);
              if (in)
                *reinterpret_cast<uint4*>(orow + (int64_t)r * a.H * D + 32 * g) =
                    make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
        }
        ++it;
      }
      } else {
        done = true;
      }
    } else {
      // ----------------------------------------------------------------- state
      // Thread = value row.  Before a chunk: the row to bf16 for QS, and times e^{G_C} back
      // into tensor memory for KV; a job's first chunk takes its initial state instead.
      const uint32_t col = lanes + kT_S;
      uint8_t* sb = sm + kSbOff + row * 128;
      int it = 0;
#pragma unroll 1
      for (int d = 0;; ++d) {
        if (!wait_warp(bRFull + (d & 1), (uint32_t)(d >> 1))) break;
        const Rec& v = recs[d & 1];
        const int len = v.len, flags = v.flags;
        const float* init = v.init;
        float* fin = (flags & kLast) ? v.fin : nullptr;
        float* decay = (flags & kLast) ? v.decay : nullptr;
        const float sofar = v.sofar, gam = exp2_approx(v.total);
        arrive(bREmpty + (d & 1));
        done = (flags & kStop) != 0;
        if (done) break;
        const bool first = (flags & kFirst) != 0;
        if (decay && row == 0) *decay = exp2_approx(sofar);
        if (init) init += row * D;
        if (fin) fin += row * D;
        if (len > 0) {
          // (a job's end waits for the state, so its KV is done where the next one begins)
          if (!first && !wait_warp(bKV, (uint32_t)it - 1)) break;
          tc_fence_after();
        }
        bool ok = true;
        // pass 0: before the chunk; pass 1: the final state, after its KV
#pragma unroll 1
        for (int pass = len > 0 ? 0 : 1; pass < 2; ++pass) {
          if (pass == 1) {
            if (!(flags & kLast)) break;
            if (len > 0) {
              ok = wait_warp(bKV, (uint32_t)it);
              if (!ok) break;
              tc_fence_after();
            }
            if (!fin) break;
          }
          const bool from_init = pass == 0 ? first : len <= 0;
#pragma unroll 1
          for (int p = 0; p < 4; ++p) {
            float x[32];
            if (from_init) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 y = init ? *reinterpret_cast<const float4*>(init + 32 * p + i)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
              }
            } else {
              tmem_ld32(col + 32 * p, x);
              tmem_wait_ld();
            }
            if (pass == 1) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(fin + 32 * p + i) =
                    make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else {
              if (kOut) {
                if (p == 0 && it > 0) {  // QS has read the copy of the chunk before
                  ok = wait_warp(bQS, (uint32_t)it - 1);
                  if (!ok) break;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint4 y = make_uint4(pack_bf16(x[8 * e], x[8 * e + 1]),
                                             pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                                             pack_bf16(x[8 * e + 4], x[8 * e + 5]),
                                             pack_bf16(x[8 * e + 6], x[8 * e + 7]));
                  *reinterpret_cast<uint4*>(sb + (p >> 1) * kHalfTile +
                                            (((4 * (p & 1) + e) ^ (row & 7)) << 4)) = y;
                }
              }
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 z = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(gam, gam));
                x[i] = z.x;
                x[i + 1] = z.y;
              }
              tmem_st32(col + 32 * p, x);
            }
          }
          if (!ok) break;
          if (pass == 0) {
            tmem_wait_st();
            tc_fence_before();
            if (kOut) fence_proxy_async_smem();
            arrive(bS);
          }
        }
        if (!ok) break;
        if (len > 0) ++it;
      }
    }
  }
  if (!done && lane == 0) atomicExch(a.err, kDevErrTimeout);  // a wait gave up
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- long chains first
// Clears the ticket counter and lists the sequences by falling length: with the longest
// drawn first the CTAs end together (186 us to the last CTA's end against a median of 158 in
// the order of cu_seqlens, 14 sequences of 1 to 4096 tokens, 48 heads).  One thread a sequence
// counts those before it.
constexpr int kMaxOrder = 1024;
__global__ void __launch_bounds__(kMaxOrder) lin_order_kernel(LinArgs a, int* ticket, int* order) {
  __shared__ int len[kMaxOrder];
  const int n = threadIdx.x;
  release_next();
  if (n == 0) *ticket = 0;
  if (n < a.n_seqs) {
    int64_t t0, t1;
    seq_range(a, n, t0, t1);
    len[n] = (int)(t1 - t0);
  }
  __syncthreads();
  if (n < a.n_seqs) {
    int before = 0;
    for (int m = 0; m < a.n_seqs; ++m) before += len[m] > len[n] || (len[m] == len[n] && m < n);
    order[before] = n;
  }
}

// ---------------------------------------------------------------------- segments
// With few chains a sequence is cut into segments of `L` chunks that run at once: a first
// pass forms every segment's end state from a zero state (the first from h0), a scan turns
// them into the states entering the segments,
//     S_in(0) = h0,   S_in(1) = S_end(0),   S_in(k+1) = S_end(k) + (segment k's decay) S_in(k),
// and the pass with outputs starts each segment from its own (also the first, so that hT
// may be h0: h0 is not read any more when a last segment writes hT).
// A malformed cu_seqlens may ask for any number of segments (sequences that overlap): the sums
// are 64 bits and what is past the table is dropped.
__global__ void __launch_bounds__(1024) lin_seg_plan_kernel(LinArgs a, int L, int4* tab,
                                                            int* first, int* n_segs, int cap,
                                                            int* tickets) {
  __shared__ int64_t warp_sums[32];
  __shared__ int64_t carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  release_next();
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
    int64_t v = P;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int64_t w = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sums[lane] = w;
    }
    __syncthreads();
    const int64_t f = carry + v - P + (warp > 0 ? warp_sums[warp - 1] : 0);
    if (n < a.n_seqs) {
      first[n] = (int)min(f, (int64_t)cap);
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
    first[a.n_seqs] = *n_segs = (int)min(carry, (int64_t)cap);
    tickets[0] = tickets[1] = 0;
  }
}

constexpr int kScanThreads = 256, kScanAhead = 8;
__global__ void __launch_bounds__(kScanThreads) lin_seg_scan_kernel(
    const int* first, int H, const float* __restrict__ h0, const float* s_end, const float* decay,
    float* s_in) {
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit - (int64_t)n * H);
  const int64_t e = 4 * ((int64_t)blockIdx.y * kScanThreads + threadIdx.x);
  wait_previous();
  release_next();
  const int f0 = first[n], f1 = first[n + 1];
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h0) s = *reinterpret_cast<const float4*>(h0 + unit * D * D + e);
  if (f0 < f1) *reinterpret_cast<float4*>(s_in + ((int64_t)f0 * H + h) * D * D + e) = s;
  for (int fb = f0; fb + 1 < f1; fb += kScanAhead) {
    float4 x[kScanAhead];
    float d[kScanAhead];
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (fb + i + 1 < f1) {
        const int64_t unit_f = (int64_t)(fb + i) * H + h;
        x[i] = *reinterpret_cast<const float4*>(s_end + unit_f * D * D + e);
        d[i] = decay[unit_f];
      }
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (fb + i + 1 < f1) {
        s = fb + i == f0 ? x[i]
                         : make_float4(fmaf(d[i], s.x, x[i].x), fmaf(d[i], s.y, x[i].y),
                                       fmaf(d[i], s.z, x[i].z), fmaf(d[i], s.w, x[i].w));
        *reinterpret_cast<float4*>(s_in + ((int64_t)(fb + i + 1) * H + h) * D * D + e) = s;
      }
  }
}

struct SegLayout {
  int4* tab;
  int *first, *n_segs, *tickets;
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
  l.n_segs = reinterpret_cast<int*>(take(3 * sizeof(int)));
  l.tickets = l.n_segs + 1;  // [2], one a pass
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
cudaError_t run(const CUtensorMap* tm, const LinArgs& a, int64_t items, bool chained,
                const char* name, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      lin_tc_kernel<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  ProfScope prof_scope(name, s);
  const dim3 grid((unsigned)(items < sms ? items : sms));
  if (chained)
    return launch_chained(lin_tc_kernel<kOut>, grid, kThreads, kSmemBytes, s, tm[0], tm[1], tm[2],
                          a);
  lin_tc_kernel<kOut><<<grid, kThreads, kSmemBytes, s>>>(tm[0], tm[1], tm[2], a);
  return cudaGetLastError();
}

}  // namespace

// Chunks of a segment, 0: sequences are not cut.  As many segments as SMs, if that pays for
// three more launches and a second trip through k and v (in segments of L chunks it takes
// about as long as 6 + 2 L uncut ones).  Uncut -> cut: one head, 6, 8, 16 and 64 chunks 24.0 ->
// 25.0, 28.8 -> 25.0, 47.8 -> 25.3 and 162 -> 32 us; 38 heads, 8 (L = 2), 12 (3), 16 (4) and 32
// (8) chunks 28.9 -> 32.9, 38.4 -> 37.0, 48.0 -> 42.2 and 86.7 -> 62.8.  Two segments (51 to 76
// chains of 152 SMs) gain what the state pass saves over a whole one: 64 heads, 32, 48, 64 and
// 128 chunks 88 -> 93, 126 -> 127, 165 -> 159 and 319 -> 287.
// The rule sees the number of sequences and their average length alone: short ones count as long
// ones do, and a long prompt packed with them may stay uncut (131072 tokens x 16 heads 0.50 ms by
// themselves, 2.46 with four one-token sequences).
int linear_segment_chunks(int64_t n_tokens, int n_seqs, int H, int forced, bool sequential) {
  if (sequential || n_tokens == 0) return 0;
  if (forced > 0) return forced;
  const int64_t sms = sm_count(), chains = (int64_t)n_seqs * H;
  if (2 * chains > sms) return 0;
  const int64_t chunks = (n_tokens / C + n_seqs) / n_seqs;  // of an average sequence
  const int64_t P = sms / chains < chunks ? sms / chains : chunks;
  const int64_t L = (chunks + P - 1) / P;
  if (chunks < (3 * chains <= sms ? 6 + 2 * L : 64)) return 0;
  return (int)L;
}

size_t linear_tc_workspace_bytes(int64_t n_tokens, int n_seqs, int H, int seg_chunks) {
  if (seg_chunks > 0) return seg_layout(nullptr, n_tokens, n_seqs, H, seg_chunks).bytes;
  return 256 + (size_t)(n_seqs < kMaxOrder ? n_seqs : kMaxOrder) * sizeof(int);
}

cudaError_t launch_linear_tc(const void* q, const void* k, const void* v, const float* g,
                             int g_head, float scale, const float* h0, const int32_t* cu,
                             int64_t T_per_seq, void* o, float* hT, int64_t n_tokens, int n_seqs,
                             int H, int Hk, int seg_chunks, void* ws, int* err, cudaStream_t s) {
  if (!err) return cudaErrorInvalidSymbol;  // the kernels report through it
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
  if (seg_chunks <= 0) {
    // Chains of different lengths, several a CTA: drawn by ticket where a chain is long enough
    // to make up for the ordering launch (in the order given -> by ticket: 2 sequences of 300
    // and 900 tokens, 96 heads 45.8 -> 37.9 us; two of 600 44.5 -> 47.4; 8 of 65 to 975, 48
    // heads 60 -> 58; 4 of 300, 96 heads 46.4 -> 48.7; from 40 chains an SM no difference).
    // Long is meant of the average: one long sequence among many short ones draws no tickets.
    const int64_t chains = (int64_t)n_seqs * H;
    if (cu && n_seqs > 1 && chains > sm_count() && n_tokens >= (int64_t)n_seqs * 4 * C) {
      a.ticket = static_cast<int*>(ws);
      if (n_seqs <= kMaxOrder) {
        int* order = a.ticket + 64;
        ProfScope prof_scope("kda_linear_order", s);
        lin_order_kernel<<<1, (unsigned)((n_seqs + 31) / 32 * 32), 0, s>>>(a, a.ticket, order);
        e = cudaGetLastError();
        a.order = order;
      } else {
        e = cudaMemsetAsync(ws, 0, sizeof(int), s);
      }
      if (e != cudaSuccess) return e;
    }
    return run<true>(tm, a, chains, a.order != nullptr, "kda_linear_tc", s);
  }
  const SegLayout l = seg_layout(ws, n_tokens, n_seqs, H, seg_chunks);
  {
    ProfScope prof_scope("kda_linear_seg_plan", s);
    lin_seg_plan_kernel<<<1, 1024, 0, s>>>(a, seg_chunks, l.tab, l.first, l.n_segs, l.cap,
                                              l.tickets);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  a.tab = l.tab;
  a.n_segs = l.n_segs;
  a.s_in = l.s_in;
  a.s_end = l.s_end;
  a.seg_decay = l.decay;
  a.ticket = l.tickets;
  e = run<false>(tm, a, (int64_t)l.cap * H, true, "kda_linear_tc_state", s);
  if (e != cudaSuccess) return e;
  {
    ProfScope prof_scope("kda_linear_seg_scan", s);
    e = launch_chained(lin_seg_scan_kernel,
                       dim3((unsigned)((int64_t)n_seqs * H), D * D / 4 / kScanThreads),
                       kScanThreads, 0, s, l.first, H, h0, l.s_end, l.decay, l.s_in);
    if (e != cudaSuccess) return e;
  }
  a.ticket = l.tickets + 1;
  return run<true>(tm, a, (int64_t)l.cap * H, true, "kda_linear_tc", s);
}

}  // namespace kda
