// Finding a CTA's or a tile's tensor in a list that a kernel has in its parameters.
#pragma once

#include <stdint.h>

namespace ra {

// The last i < n with first[i] <= x, by the whole warp: first[] ascends, first[0] = 0, n <= 1024. Two rounds of
// 32 probes, against the ten dependent constant loads of a bisection.
__device__ __forceinline__ int last_not_above(const uint32_t* first, int n, uint32_t x) {
  if (n == 1) return 0;
  const int lane = threadIdx.x & 31, step = (n + 31) / 32;
  int i = lane * step;
  int lo = (__popc(__ballot_sync(0xffffffffu, i < n && first[i] <= x)) - 1) * step;
  i = lo + lane;
  return lo + __popc(__ballot_sync(0xffffffffu, lane < step && i < n && first[i] <= x)) - 1;
}

}  // namespace ra
