// Drafted trees on the device, shared by the kernels that take them.
#pragma once

#include "device_common.h"

namespace nvfp4 {

// Ancestor-or-self bits of node v of a tree of at most 64 nodes, lane = node:
// parent pointers doubled six times.  A parent outside [0, v) makes v a root.
// add(at, on): what lane `at` has gathered along its line belongs to this one's, too,
// where `on`.
template <typename Add>
__device__ __forceinline__ uint64_t ancestors_of_wave(int par, Add add) {
  const int lane = threadIdx.x & 63;
  uint64_t mask = 1ull << lane;
  int p = par >= 0 && par < lane ? par : -1;
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const int at = p < 0 ? lane : p;
    const uint64_t up = __shfl(mask, at);
    const int pp = __shfl(p, at);
    add(at, p >= 0);
    if (p >= 0) {
      mask |= up;
      p = pp;
    }
  }
  return mask;
}

__device__ __forceinline__ uint64_t ancestors_of_wave(int par) {
  return ancestors_of_wave(par, [](int, bool) {});
}

}  // namespace nvfp4
