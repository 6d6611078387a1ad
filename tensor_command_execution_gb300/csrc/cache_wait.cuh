// cache_wait.cuh - a wait that ends: on a barrier, or because it took too long.
// (Plain C++ too: its rules are tested on the host.)
#pragma once

#include <cstdint>

#ifndef __CUDACC__
#define __device__
#define __forceinline__ inline
#endif

namespace cmdx {

constexpr uint64_t kPatience = 2000000000;  // ns: no wait takes longer

// Whether `ready` said yes. A wait that takes longer than kPatience gives up for
// the whole CTA, whose word it sets; one that finds the word set gives up soon.
// (Clock and word are looked at now and then only: a look takes about as long as
// a wait should.)
template <class Ready, class Now>
__device__ __forceinline__ bool wait_until(volatile uint32_t* stop, Ready ready, Now now) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !ready(); ++n) {
    if (n % 256) continue;
    if (*stop) return false;
    const uint64_t t = now();
    if (t0 == 0) t0 = t;
    if (t - t0 > kPatience) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// ... whatever the word says: for what this CTA has on its way, before it ends.
template <class Ready, class Now>
__device__ __forceinline__ bool wait_anyway(volatile uint32_t* stop, Ready ready, Now now) {
  uint32_t mine = 0;
  const bool ok = wait_until(&mine, ready, now);
  if (!ok) *stop = 1;
  return ok;
}

}  // namespace cmdx
