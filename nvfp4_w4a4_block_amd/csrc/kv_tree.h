// Drafted trees on the device, shared by the kernels that take them.
#pragma once

#include "device_common.h"

namespace nvfp4 {

// Ancestor-or-self bits of node v of a tree of at most 64 nodes, lane = node:
// parent pointers doubled six times.  A parent outside [0, v) makes v a root.
__device__ __forceinline__ uint64_t ancestors_of_wave(int par) {
  const int lane = threadIdx.x & 63;
  uint64_t mask = 1ull << lane;
  int p = par >= 0 && par < lane ? par : -1;
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const int at = p < 0 ? lane : p;
    const uint64_t up = __shfl(mask, at);
    const int pp = __shfl(p, at);
    if (p >= 0) {
      mask |= up;
      p = pp;
    }
  }
  return mask;
}

}  // namespace nvfp4
