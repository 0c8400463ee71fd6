// Token and target numbers of 32 or 64 bits.
#pragma once

#include <stdint.h>

namespace ra {

struct Indices {
  const void* p;
  int size;  // bytes each: 4 or 8
};
__device__ __forceinline__ int64_t load_index(const Indices& a, uint64_t i) {
  return a.size == 4 ? (int64_t) static_cast<const int32_t*>(a.p)[i] : static_cast<const int64_t*>(a.p)[i];
}

}  // namespace ra
