// Host-side helpers shared by the translation units behind the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ra.h"

namespace ra {

// Records `err` for ra_last_cuda_error() and returns RA_ERR_CUDA.
ra_status_t cuda_failed(cudaError_t err);

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi) in bytes; empty if lo == hi
};
inline bool overlaps(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// A launch's status: success, or the CUDA error recorded.
inline ra_status_t launched(cudaError_t err) { return err == cudaSuccess ? RA_SUCCESS : cuda_failed(err); }

// Bytes of an element of the floating types; 0 for any other code.
inline int float_size(int dtype) {
  return dtype == RA_FLOAT32 ? 4 : (dtype == RA_FLOAT16 || dtype == RA_BFLOAT16) ? 2 : 0;
}
// The status of a dtype that an operator on floating types is given.
inline ra_status_t check_float(int dtype) {
  return float_size(dtype) ? RA_SUCCESS : dtype == RA_INT32 ? RA_ERR_UNSUPPORTED : RA_ERR_INVALID_ARG;
}

}  // namespace ra
