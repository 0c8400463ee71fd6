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

// Bytes from a matrix's first element to past its last.
inline uint64_t extent(uint64_t rows, uint64_t cols, uint64_t stride, uint64_t es) { return ((rows - 1) * stride + cols) * es; }

// One buffer of a call.
struct Buffer {
  const void* p;
  uint64_t bytes;
  uintptr_t align;
  bool needed;
  Range at;
  uint64_t stride = 0;  // of a matrix, in bytes
};

// A span of 2^57 elements at most, not null (unless it may be), aligned, inside the address space.
inline bool sound(Buffer& b) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(b.p);
  b.at = {};
  if (lo == 0) return !b.needed;
  if (lo % b.align || lo + b.bytes < lo) return false;
  b.at = {lo, lo + (uintptr_t)b.bytes};
  return true;
}
// Whether two buffers share a byte. Matrices of one stride whose rows (of `width` bytes) lie side by side do not, as
// column slices of one matrix.
inline bool shares(const Buffer& a, const Buffer& b, uint64_t width) {
  if (!overlaps(a.at, b.at)) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  const uint64_t apart = (a.at.lo < b.at.lo ? b.at.lo - a.at.lo : a.at.lo - b.at.lo) % a.stride;
  return apart < width || apart + width > a.stride;
}
inline bool shape_ok(uint64_t rows, uint64_t cols) {
  return rows <= RA_MAX_COUNT && cols <= RA_MAX_COUNT && (cols == 0 || rows <= RA_MAX_COUNT / cols);
}
inline bool stride_ok(uint64_t rows, uint64_t cols, uint64_t stride) {
  return stride >= cols && stride <= RA_MAX_COUNT && (stride == 0 || rows <= RA_MAX_COUNT / stride);
}

}  // namespace ra
