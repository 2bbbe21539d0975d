// kda_scan.cu -- selective state space scan over packed sequences: for every channel c with
// states s = 0 .. S-1 (S = 8, 16, 32) and delta_t = softplus(dt_t + bias),
//     h_t[s] = exp(delta_t A[s]) h_{t-1}[s] + delta_t x_t B_t[s]
//     y_t    = (sum_s C_t[s] h_t[s] + D x_t) SiLU(z_t)
// B and C are shared by the channels of a group.  The states are fp32.
//
// A CTA takes 256 / S neighbouring channels of one sequence.  Its warps take tiles of 8 tokens in
// turn and pass the state round a ring.  What a tile does to a state is known before the state
// comes: with own_t the states from zero, all_t the products of the decays and time the sum of the
// steps,
//     h_out = exp(A time) h_in + own_8,   y_t = C_t . own_t + (C_t all_t) . h_in,
// so a warp forms all of that ahead (a lane holds 8 states of one channel, S / 8 lanes share a
// channel, the 64 products C_t all_t stay in its registers), and what is serial is one product and
// sum a tile on its way from warp to warp.  Outputs and the next tile's steps follow behind that.
//
// Bound by what the schedulers can issue: a state, token and channel takes 7 fp32 operations (4 in
// the plain recurrence) and one exponential, a token and channel some 45 instructions for its step,
// its gate and its copies, and packed operations, two at once, take two turns of the lanes that
// integer instructions use too.  8192 tokens x 8192 channels of 16 states, bf16: 418 us, 117 ns a tile
// and SM, 67% of the issue slots (38% of the exponentials', 19% of HBM); 65536 x 2048: 889 us; fp32 8192 x
// 4096: 235 us.  In the first case with a CTA a unit (452 us, 111 ns a tile, four rounds instead of three
// and a half): the bare recurrence (4 operations, handed on behind them) 456 us, and 2.1 times as long
// with 2048 channels; scalar instead of packed operations 557 us; inputs that wait in registers instead
// of shared memory 680 us (a load in flight holds one of the few scoreboards that the code between
// needs).
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

#include "kda_internal.cuh"
#include "kda_scan.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kTok = 8;  // tokens of a tile

// The halves of a cluster's barrier.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
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

// A lane's eight states, kept by lanes.
__device__ __forceinline__ void put_state(float4 (*s)[32], int lane, const float2 (&h)[4]) {
  s[0][lane] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  s[1][lane] = make_float4(h[2].x, h[2].y, h[3].x, h[3].y);
}
__device__ __forceinline__ void get_state(const float4 (*s)[32], int lane, float2 (&h)[4]) {
  const float4 lo = s[0][lane], hi = s[1][lane];
  h[0] = make_float2(lo.x, lo.y); h[1] = make_float2(lo.z, lo.w);
  h[2] = make_float2(hi.x, hi.y); h[3] = make_float2(hi.z, hi.w);
}
__device__ __forceinline__ void get_last(const float2 (&h)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = h[i].x;
    v[2 * i + 1] = h[i].y;
  }
}

// Shared memory of a warp.  Rows of a tile are looked after by four lanes each (kVec channels a
// lane); states belong to lanes by channel and eighth, lane = channel + kCh * eighth.
template <typename T, int kS>
struct ScanWarp {
  static constexpr int kLn = kS / 8, kCh = 32 / kLn, kVec = kCh / 4;
  static constexpr int kX = kVec * (int)sizeof(T) / 4, kB = kS * (int)sizeof(T) / 8;  // words a lane
  __align__(16) uint32_t x[32][kX], dt[32][kX], z[32][kX], bc[32][kB];  // a tile as it comes
  __align__(16) float delta[2][kTok][kCh];  // of this tile and the next
  __align__(16) float dx[2][kTok][kCh];     // delta x
  __align__(16) float BC[2][2][kTok][kS];
  __align__(16) float part[kLn][(kTok + 1) * kCh];  // sums over a lane's states (a row to spare:
                                                    // other banks for every eighth)
  __align__(16) float4 state[2][32];        // what the warp hands on
};

// kN consecutive elements of T as they lie in memory.
template <typename T, int kN>
struct Raw {
  static constexpr int kWords = kN * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  // By way of the lane's own piece of shared memory: nothing of a tile in flight sits in registers
  // (whose few scoreboards the code in between needs).
  static __device__ __forceinline__ void copy(uint32_t* to, const char* p, bool valid) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (kWords < 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(p),
                   "n"(4 * kWords), "r"(valid ? 4 * kWords : 0)
                   : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + 4 * i),
                     "l"(p + 4 * i), "r"(valid ? 16 : 0)
                     : "memory");
    }
  }
  __device__ __forceinline__ void take(const uint32_t* from) {
    if constexpr (kWords == 1) {
      w[0] = *from;
    } else if constexpr (kWords == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(from);
      w[0] = u.x; w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(from + i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {  // elements 2 i and 2 i + 1
    if constexpr (sizeof(T) == 2)
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ void set_pair(int i, float2 v) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  __device__ __forceinline__ void store(char* p) const {
    if constexpr (kWords == 1) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
};
// kN floats (2, 4 or 8) in shared memory.
template <int kN>
__device__ __forceinline__ void put(float* p, const float2* v) {
  if constexpr (kN == 2) {
    *reinterpret_cast<float2*>(p) = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
  }
}
template <int kN>
__device__ __forceinline__ void get(const float* p, float2* v) {
  if constexpr (kN == 2) {
    v[0] = *reinterpret_cast<const float2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
      const float4 u = reinterpret_cast<const float4*>(p)[i];
      v[2 * i] = make_float2(u.x, u.y);
      v[2 * i + 1] = make_float2(u.z, u.w);
    }
  }
}

// What a segment of a sequence does to a state (kCut): h -> exp(A time) h + own.
template <int kS>
struct Segment {
  float4 own[2][32];
  float time[256 / kS];
};

// How the work is drawn: a unit (some neighbouring channels of one sequence) a CTA; or the CTAs of a
// cluster take a segment of its sequence each, two passes over it: what it does to a state, then, from
// the state that the segments before it leave, the scan; or two CTAs share several units.
enum How { kUnits, kSegments, kPairs };
enum Piece { kWhole, kFirstHalf, kSecondHalf };  // of a unit

// A unit (or what of it is this CTA's) by a ring of kWarps.
template <typename T, int kS, int kWarps, How kHow>
__device__ __forceinline__ void scan_unit(const ScanArgs& a, int* err, char* smem, int unit,
                                          Piece piece) {
  using W = ScanWarp<T, kS>;
  constexpr bool kCut = kHow == kSegments, kPair = kHow == kPairs;
  constexpr int kLn = W::kLn, kCh = W::kCh, kVec = W::kVec, kBc = kS / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  W& w = reinterpret_cast<W*>(smem)[warp];
  const int from = (warp + kWarps - 1) % kWarps;
  const W& before = reinterpret_cast<W*>(smem)[from];

  const int per_group = a.C / a.G;
  const int blocks = (per_group + kCh - 1) / kCh;  // of a group
  cg::cluster_group cluster = cg::this_cluster();  // (of one CTA, a unit a CTA)
  __shared__ float4 enter[2][32];                  // the state that comes from another CTA
  const int n = unit / (blocks * a.G), rest = unit - n * (blocks * a.G);
  const int g = rest / blocks, first = (rest - g * blocks) * kCh;  // first channel in the group
  int64_t t0, t1;
  if (!seq_range(a, n, t0, t1) && threadIdx.x == 0 && err) atomicExch(err, kDevErrBadSeqlens);
  const int cl = lane % kCh, sub = lane / kCh;
  const int width = min(kCh, per_group - first);  // channels there are (a multiple of 8)
  const bool on = cl < width;
  const int c0 = g * per_group + first, c = c0 + (on ? cl : 0);
  float2 A[4];
  {
    float v[8];
    load8(a.A + (int64_t)c * kS + 8 * sub, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] = make_float2(kLog2e * v[2 * i], kLog2e * v[2 * i + 1]);
  }
  const int64_t at = ((int64_t)n * a.C + c) * kS + 8 * sub;

  if constexpr (kCut) {
    const int64_t all = (t1 - t0 + kTok - 1) / kTok;
    const int64_t part = (all + cluster.num_blocks() - 1) / cluster.num_blocks() * kTok;
    t0 = min(t1, t0 + cluster.block_rank() * part);
    t1 = min(t1, t0 + part);
  }
  if constexpr (kPair) {
    const int64_t middle = t0 + (t1 - t0 + kTok - 1) / kTok / 2 * kTok;
    if (piece == kFirstHalf) t1 = middle;
    if (piece == kSecondHalf) t0 = middle;
  }
  const int len = (int)(t1 - t0), tiles = (len + kTok - 1) / kTok;
  if constexpr (!kCut) {
    if (tiles == 0 && warp == 0) {  // (of halves the first one, or both)
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a.h0 ? a.h0[at + i] : 0.f;
      if (kPair && piece == kFirstHalf) {
        float2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = make_float2(v[2 * i], v[2 * i + 1]);
        put_state(cluster.map_shared_rank(enter, 1), lane, h);
      } else if (a.hT && on) {
        store8(a.hT + at, v);
      }
    }
    if (warp >= tiles) return;
  }
  // The lane's part of a tile's rows: kVec channels of token `row`, and kS / 2 values of B or C.
  const int row = lane / 4, ch = kVec * (lane % 4);
  const bool has = ch < width;
  const int mine = c0 + (has ? ch : 0);
  const int64_t first_row = t0 + warp * kTok + row;
  const char* xp = static_cast<const char*>(a.x) + (first_row * a.sx + mine) * (int)sizeof(T);
  const char* dp = static_cast<const char*>(a.dt) + (first_row * a.sdt + mine) * (int)sizeof(T);
  const char* zp =
      a.z ? static_cast<const char*>(a.z) + (first_row * a.sz + mine) * (int)sizeof(T) : nullptr;
  char* yp = static_cast<char*>(a.y) + (first_row * a.sy + mine) * (int)sizeof(T);
  const int brow = (lane & 15) / 2, bcol = kBc * (lane & 1);
  const int64_t sb = lane < 16 ? a.sB : a.sC;
  const char* bp = static_cast<const char*>(lane < 16 ? a.B : a.Cm) +
                   ((t0 + warp * kTok + brow) * sb + g * kS + bcol) * (int)sizeof(T);
  constexpr int64_t kHop = (int64_t)kWarps * kTok * sizeof(T);
  float2 bias[kVec / 2], skip[kVec / 2];
#pragma unroll
  for (int j = 0; j < kVec / 2; ++j) {
    bias[j] = a.bias ? *reinterpret_cast<const float2*>(a.bias + mine + 2 * j) : both(0.f);
    skip[j] = a.D ? *reinterpret_cast<const float2*>(a.D + mine + 2 * j) : both(0.f);
  }
  const char* safe = static_cast<const char*>(a.x);  // (nothing is read from it)
  Raw<T, kVec> x, z;  // of the tile at hand
  Raw<T, kBc> rb;
  auto fetch = [&](int left) {  // `left`: tokens of the sequence from the tile's first on
    const bool ok = has && row < left;
    Raw<T, kVec>::copy(w.x[lane], ok ? xp : safe, ok);
    Raw<T, kVec>::copy(w.dt[lane], ok ? dp : safe, ok);
    if (zp) Raw<T, kVec>::copy(w.z[lane], ok ? zp : safe, ok);
    Raw<T, kBc>::copy(w.bc[lane], brow < left ? bp : safe, brow < left);
    xp += kHop * a.sx;
    dp += kHop * a.sdt;
    zp += zp ? kHop * a.sz : 0;
    bp += kHop * sb;
  };
  // Steps of the fetched tile, and its B and C as fp32: in registers, then in shared memory.
  float2 fd[kVec / 2], fx[kVec / 2];
  auto front = [&](int left) {
    Raw<T, kVec> rd;
    x.take(w.x[lane]);
    z.take(w.z[lane]);  // (whatever lies there, without a gate)
    rd.take(w.dt[lane]);
    rb.take(w.bc[lane]);
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      fd[j] = __fadd2_rn(rd.pair(j), bias[j]);
      const float2 sp = softplus2(fd[j]);
      if (a.softplus) fd[j] = sp;
      if (row >= left) fd[j] = both(0.f);  // behind the end: the state stays
      fx[j] = __fmul2_rn(fd[j], x.pair(j));
    }
  };
  auto lay = [&](int buf) {
    put<kVec>(&w.delta[buf][row][ch], fd);
    put<kVec>(&w.dx[buf][row][ch], fx);
    float2 v[kBc / 2];
#pragma unroll
    for (int j = 0; j < kBc / 2; ++j) v[j] = rb.pair(j);
    put<kBc>(&w.BC[buf][lane / 16][brow][bcol], v);
  };
  // The state that comes in from outside, and what leaves at the end (of an uncut sequence at once).
  __shared__ Segment<kS> mine_seg;
  __shared__ float times[kWarps][kCh];
  float last[8];
  bool ends = false;
  auto outside = [&](float2 (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = a.h0 ? *reinterpret_cast<const float2*>(a.h0 + at + 2 * i) : both(0.f);
  };
  auto start = [&] {  // the first tile's front, the second one's copies
    fetch(len - warp * kTok);
    wait_copies();
    front(len - warp * kTok);
    lay(0);
    __syncwarp();
    if (warp + kWarps < tiles) fetch(len - (warp + kWarps) * kTok);
  };
  if constexpr (kCut) {
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    float sum = 0.f;
    if (rank + 1 < ctas && warp < tiles) {  // (nothing follows on the last segment)
      const char *const x0 = xp, *const d0 = dp, *const z0 = zp, *const b0 = bp;
      zp = nullptr;
      start();
      int buf = 0;
      for (int tile = warp; tile < tiles; tile += kWarps) {
        float2 own[4], h[4];
        float time = 0.f;
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
          const float d = w.delta[buf][t][cl], dx = w.dx[buf][t][cl];
          float2 bs[4];
          get<8>(&w.BC[buf][0][t][8 * sub], bs);
          time += d;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = __fmul2_rn(A[i], both(d));
            const float2 add = __fmul2_rn(both(dx), bs[i]);
            own[i] = t == 0 ? add : __ffma2_rn(make_float2(ex2(u.x), ex2(u.y)), own[i], add);
          }
        }
        sum += time;
        if (tile > 0) {
          handed(1 + from);
          get_state(before.state, lane, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = __fmul2_rn(A[i], both(time));
            own[i] = __ffma2_rn(make_float2(ex2(u.x), ex2(u.y)), h[i], own[i]);
          }
        }
        if (tile + 1 < tiles) {
          put_state(w.state, lane, own);
          hand(1 + warp);
        } else {
          put_state(mine_seg.own, lane, own);
        }
        wait_copies();
        front(len - (tile + kWarps) * kTok);
        buf ^= 1;
        lay(buf);
        __syncwarp();
        if (tile + 2 * kWarps < tiles) fetch(len - (tile + 2 * kWarps) * kTok);
      }
      xp = x0; dp = d0; zp = z0; bp = b0;
    }
    if (sub == 0) times[warp][cl] = sum;
    __syncthreads();
    if (warp == 0 && sub == 0) {
      float time = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) time += times[i][cl];
      mine_seg.time[cl] = time;
    }
    if (warp == 0 && tiles == 0) {
      const float2 none[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
      put_state(mine_seg.own, lane, none);
    }
    __syncwarp();
    cluster.sync();
    if (warp == 0) {
      float2 h[4];
      outside(h);
#pragma unroll 1
      for (int j = 0; j < rank; ++j) {
        const Segment<kS>* seg = cluster.map_shared_rank(&mine_seg, j);
        const float time = seg->time[cl];
        float2 own[4];
        get_state(seg->own, lane, own);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = __fmul2_rn(A[i], both(time));
          h[i] = __ffma2_rn(make_float2(ex2(u.x), ex2(u.y)), h[i], own[i]);
        }
      }
      put_state(enter, lane, h);
      __syncwarp();
      if (tiles == 0 && rank + 1 == ctas) {
        ends = true;
        get_last(h, last);
      }
    }
    cluster_arrive();  // outside and segments are read
  }
  if (!kCut || warp < tiles) {
    start();
    int buf = 0;
    for (int tile = warp; tile < tiles; tile += kWarps) {
      const int left = len - tile * kTok;  // tokens from the tile's first on
      // what the tile's tokens do to a state that comes in: h -> all h + own, y = acc + share . h
      float2 own[4], all[4], share[kTok][4];
      float acc[kTok], time = 0.f;
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        const float d = w.delta[buf][t][cl], dx = w.dx[buf][t][cl];
        float2 bs[4], cs[4];
        get<8>(&w.BC[buf][0][t][8 * sub], bs);
        get<8>(&w.BC[buf][1][t][8 * sub], cs);
        time += d;
        float2 y2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = __fmul2_rn(A[i], both(d));
          const float2 e = make_float2(ex2(u.x), ex2(u.y));
          const float2 add = __fmul2_rn(both(dx), bs[i]);
          own[i] = t == 0 ? add : __ffma2_rn(e, own[i], add);
          all[i] = t == 0 ? e : __fmul2_rn(e, all[i]);
          y2 = i == 0 ? __fmul2_rn(cs[i], own[i]) : __ffma2_rn(cs[i], own[i], y2);
          share[t][i] = __fmul2_rn(cs[i], all[i]);
        }
        acc[t] = y2.x + y2.y;
      }
      // (the state itself decays by one exponential a tile: their errors, of about 2^-26 and one
      // sign, add up over as many tokens as a slow decay remembers)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = __fmul2_rn(A[i], both(time));
        all[i] = make_float2(ex2(u.x), ex2(u.y));
      }
      float2 h[4];
      if (tile > 0) {
        handed(1 + from);
        get_state(before.state, lane, h);
      } else if constexpr (kCut) {
        get_state(enter, lane, h);
      } else if (kPair && piece == kSecondHalf) {
        get_state(enter, lane, h);
      } else {
        outside(h);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = __ffma2_rn(all[i], h[i], own[i]);
      if (tile + 1 < tiles) {
        put_state(w.state, lane, own);
        hand(1 + warp);
      } else {
        get_last(own, last);
        if constexpr (kCut)
          ends = cluster.block_rank() + 1 == cluster.num_blocks();
        else if (kPair && piece == kFirstHalf)
          put_state(cluster.map_shared_rank(enter, 1), lane, own);
        else if (a.hT && on)
          store8(a.hT + at, last);
      }
      // this tile's outputs, and the next one's front between them (of zeros, behind the last)
      float2 gate[kVec / 2], old[kVec / 2];
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) {
        old[j] = __fmul2_rn(skip[j], x.pair(j));
        gate[j] = silu2(z.pair(j));
        if (!a.z) gate[j] = both(1.f);
      }
      wait_copies();
      front(left - kWarps * kTok);
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        float2 y2 = __fmul2_rn(share[t][0], h[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) y2 = __ffma2_rn(share[t][i], h[i], y2);
        acc[t] += y2.x + y2.y;
      }
      buf ^= 1;
#pragma unroll
      for (int t = 0; t < kTok; ++t) w.part[sub][t * kCh + cl] = acc[t];
      lay(buf);
      __syncwarp();
      if (tile + 2 * kWarps < tiles) fetch(len - (tile + 2 * kWarps) * kTok);
      float2 v[kVec / 2];
      get<kVec>(&w.part[0][row * kCh + ch], v);
#pragma unroll
      for (int m = 1; m < kLn; ++m) {
        float2 u[kVec / 2];
        get<kVec>(&w.part[m][row * kCh + ch], u);
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) v[j] = __fadd2_rn(v[j], u[j]);
      }
      Raw<T, kVec> out;
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j)
        out.set_pair(j, __fmul2_rn(__fadd2_rn(v[j], old[j]), gate[j]));
      if (has && row < left) out.store(yp);
      yp += kHop * a.sy;
      __syncwarp();  // the sums have been read
    }
  }
  if constexpr (kCut) {
    cluster_wait();
    if (ends && a.hT && on) store8(a.hT + at, last);  // (hT may be h0)
  }
}

// kWarps: 12 of them an SM in one CTA or in three of 4.
template <typename T, int kS, int kWarps, How kHow>
__global__ void __launch_bounds__(32 * kWarps, 12 / kWarps) scan_kernel(const ScanArgs a, int* err) {
  extern __shared__ __align__(16) char smem[];
  if constexpr (kHow != kPairs) {
    const int ctas = kHow == kSegments ? (int)cg::this_cluster().num_blocks() : 1;
    scan_unit<T, kS, kWarps, kHow>(a, err, smem, (int)blockIdx.x / ctas, kWhole);
  } else {
    // Every so many-th unit is a pair's (neighbours run at the same time: their rows lie beside each
    // other), the first half of them the first CTA's and the rest the second's; the middle one of
    // an odd number is cut: the first CTA begins with its half, the second ends with its own, for
    // which the state has long been there.
    constexpr int kCh = ScanWarp<T, kS>::kCh;
    const int units = a.N * a.G * ((a.C / a.G + kCh - 1) / kCh);
    const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2, rank = (int)blockIdx.x % 2;
    const int count = units / pairs + (pair < units % pairs), pieces = (count + 1) / 2;
    const int first = pair + pairs * (rank * (count / 2));
    cg::this_cluster().sync();  // the other CTA is there
    const bool odd = count % 2 != 0, gives = odd && rank == 0;
    if (!gives) cluster_arrive();
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      Piece piece = kWhole;
      if (gives && i == 0) piece = kFirstHalf;
      if (odd && rank == 1 && i + 1 == pieces) {
        cluster_wait();  // the state is there
        piece = kSecondHalf;
      }
      const int unit = first + pairs * ((rank == 0 ? i + pieces - 1 : i + 1) % pieces);
      scan_unit<T, kS, kWarps, kHow>(a, err, smem, unit, piece);
      __syncthreads();  // the ring is at rest
      if (gives && i == 0) cluster_arrive();
    }
    if (!odd || rank == 0) cluster_wait();
  }
}

template <typename T, int kS, int kWarps, How kHow>
cudaError_t launch_scan_t(const ScanArgs& a, unsigned units, int ctas, int* err, cudaStream_t s) {
  constexpr size_t smem = kWarps * sizeof(ScanWarp<T, kS>);
  const auto kernel = scan_kernel<T, kS, kWarps, kHow>;
  static std::atomic<uint64_t> told{0};  // devices that know how much shared memory this takes
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(told.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    told |= bit;
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(units * (unsigned)ctas);
  c.blockDim = dim3(32 * kWarps);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = kHow == kUnits ? 0 : 1;
  return cudaLaunchKernelEx(&c, kernel, a, err);
}

int sm_count() {
  int sms = 152, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Whether three rings of 4 warps an SM are expected to end before one of 12.  A ring of 12 takes
// 117 ns a tile, one of 4 takes 200 alone, 265 beside another and 330 beside two, and a CTA some 3 us
// to begin and end, which others cover where there are any.  (512 units of 1024 tiles: 457 us by
// rings of 12, 522 by rings of 4; 2048 of 64: 136 and 116; 4096 of 64: 279 and 220.)  These hold for 16
// states and up to some 128 tiles.  At 1024 tiles one of 4 takes 216, 263 and 377: with 400 units the
// rule is 12% off (385 us by rings of 4, 345 by rings of 12), with 2048 3%.  There, with 8, 16 and 32
// states, a ring of 12 takes 135, 117 and 139 (fp32 150, 117 and 169), and rings of 4 take 1.8, 1.9 and
// 1.3 times as long alone, 2.3, 2.2 and 2.1 beside another and 3.2, 3.2 and 3.0 beside two.
bool short_rings(int64_t units, int64_t tiles, int sms, double rounds_of_12) {
  const double t = (double)tiles, one = t * 0.117 + 3;
  const int64_t rounds = units / (3 * sms), rest = units - rounds * 3 * sms;
  const double last = rest == 0 ? 0 : (rest > 2 * sms ? 0.33 : rest > sms ? 0.265 : 0.2) * t + 3;
  return rounds * (t * 0.33 + 1) + last < rounds_of_12 * one;
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, int bf16, int S, int* err, cudaStream_t s) {
  const int ch = 256 / S;
  const int64_t units = (int64_t)a.N * a.G * ((a.C / a.G + ch - 1) / ch);
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  ProfScope prof_scope("kda_scan", s);
  const int64_t tiles = (a.NT / a.N + kTok - 1) / kTok;  // of a sequence, on average
  const int sms = sm_count();
  // Few units of long sequences: a cluster each, its CTAs a segment each.  The pass that finds
  // what a segment does to a state takes about as long as its scan, so two segments gain next to
  // nothing (8192 tokens x 1024 channels 122 -> 110 us on one GPU, 119 -> 120 on another; 1024 tokens
  // lose), four halve the time (x 512 channels 119 to 121 -> 62 to 66 us,
  // 2048 tokens 38 -> 26), eight take a third (x 128 channels 119 -> 39 us).  A cluster lies within one
  // GPC, so fewer of them run at once than SMs / CTAs: 16 units and more by eights and 37 and more by
  // fours take two turns (16 to 19 units of 8192 tokens 70 us, by fours 65; 37 and 38 123 us, uncut 119).
  int cut = 1;
  while (cut < 8 && units * cut * 2 <= sms && tiles >= 128 * cut) cut *= 2;
  if (cut == 2 && tiles < 512) cut = 1;
  // Rounds of rings of 12, and those that pairs of CTAs take, which can end on half a unit (8192
  // tokens x 8192 channels 452 -> 418 us, 4096 x 2560 119 -> 96, 2048 x 5120 97 -> 84).
  const int64_t pairs = sms / 2, alone = (units + sms - 1) / sms;
  const double paired = 0.5 * (double)((units + pairs - 1) / pairs);
  const bool pair = cut == 1 && (!a.cu || a.N == 1) && units > sms && paired < alone;
  const bool four = cut == 1 && short_rings(units, tiles, sms, pair ? paired : alone);
  cudaError_t e = cudaSuccess;
  with_states(S, [&](auto k) {
    constexpr int kS = decltype(k)::value;
    using H = __nv_bfloat16;
    const auto fn =
        cut > 1 ? (bf16 ? launch_scan_t<H, kS, 12, kSegments> : launch_scan_t<float, kS, 12, kSegments>)
        : four  ? (bf16 ? launch_scan_t<H, kS, 4, kUnits> : launch_scan_t<float, kS, 4, kUnits>)
        : pair  ? (bf16 ? launch_scan_t<H, kS, 12, kPairs> : launch_scan_t<float, kS, 12, kPairs>)
                : (bf16 ? launch_scan_t<H, kS, 12, kUnits> : launch_scan_t<float, kS, 12, kUnits>);
    const bool two = pair && !four;
    e = fn(a, (unsigned)(two ? pairs : units), two ? 2 : cut, err, s);
  });
  return e;
}

}  // namespace kda
