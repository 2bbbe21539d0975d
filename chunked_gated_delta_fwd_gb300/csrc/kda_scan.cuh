// kda_scan.cuh -- what the selective scan over prompts and the one over new tokens share.
#pragma once

#include <type_traits>

#include "kda_internal.cuh"
#include "kda_layer_math.cuh"

namespace kda {

// f(integral_constant<S>) for a number of states that the entry points let through.
template <typename F>
void with_states(int S, F f) {
  if (S == 8) f(std::integral_constant<int, 8>{});
  else if (S == 16) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

// The tokens [t0, t1) of sequence n.  Offsets that do not run upwards from 0 to NT give some
// range within [0, NT]; the result says whether what this sequence shows of them is sound.
__device__ __forceinline__ bool seq_range(const ScanArgs& a, int n, int64_t& t0, int64_t& t1) {
  if (!a.cu) {
    t0 = n * a.T;
    t1 = t0 + a.T;
    return true;
  }
  const int64_t b = __ldg(a.cu + n), e = __ldg(a.cu + n + 1);
  t0 = b < 0 ? 0 : (b > a.NT ? a.NT : b);
  t1 = e < t0 ? t0 : (e > a.NT ? a.NT : e);
  return t0 == b && t1 == e && (n > 0 || b == 0) && (n < a.N - 1 || e == a.NT);
}

}  // namespace kda
