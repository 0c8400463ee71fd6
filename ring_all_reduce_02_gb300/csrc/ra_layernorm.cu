// ra_layernorm_forward / _backward: argument checks, overlap rules, launch shapes.
#include <math.h>

#include "ra_host.h"
#include "ra_layernorm.cuh"

namespace ra {
#define RA_DECLARE_LN(DT, W)                                        \
  cudaError_t ln_forward_##DT##_##W(const LnForward& a, cudaStream_t s);   \
  cudaError_t ln_backward_##DT##_##W(LnBackward a, cudaStream_t s);
RA_DECLARE_LN(0, 0)
RA_DECLARE_LN(1, 0)
RA_DECLARE_LN(1, 1)
RA_DECLARE_LN(2, 0)
RA_DECLARE_LN(2, 2)
}  // namespace ra

namespace {

using ra::Range;

using ra::kLnMaxParts;

// Bytes from a matrix's first element to past its last.
uint64_t extent(uint64_t rows, uint64_t cols, uint64_t stride, uint64_t es) { return ((rows - 1) * stride + cols) * es; }

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
bool sound(Buffer& b) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(b.p);
  b.at = {};
  if (lo == 0) return !b.needed;
  if (lo % b.align || lo + b.bytes < lo) return false;
  b.at = {lo, lo + (uintptr_t)b.bytes};
  return true;
}
// Whether two buffers share a byte. Matrices of one stride whose rows (of `width` bytes) lie side by side do not, as
// column slices of one matrix.
bool shares(const Buffer& a, const Buffer& b, uint64_t width) {
  if (!ra::overlaps(a.at, b.at)) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  const uint64_t apart = (a.at.lo < b.at.lo ? b.at.lo - a.at.lo : a.at.lo - b.at.lo) % a.stride;
  return apart < width || apart + width > a.stride;
}
bool shape_ok(uint64_t rows, uint64_t cols) {
  return rows <= RA_MAX_COUNT && cols <= RA_MAX_COUNT && (cols == 0 || rows <= RA_MAX_COUNT / cols);
}
bool stride_ok(uint64_t rows, uint64_t cols, uint64_t stride) {
  return stride >= cols && stride <= RA_MAX_COUNT && (stride == 0 || rows <= RA_MAX_COUNT / stride);
}
ra_status_t check_types(int dtype, int weight_dtype) {
  ra_status_t st = ra::check_float(dtype);
  if (st == RA_SUCCESS) st = ra::check_float(weight_dtype);
  if (st == RA_SUCCESS && weight_dtype != dtype && weight_dtype != RA_FLOAT32) st = RA_ERR_UNSUPPORTED;
  return st;
}
}  // namespace

extern "C" {

ra_status_t ra_layernorm_forward(const void* x, size_t x_stride, const void* weight, const void* bias, void* y,
                                 size_t y_stride, float* mean, float* rstd, size_t rows, size_t cols, double eps,
                                 ra_dtype_t dtype, ra_dtype_t weight_dtype, void* stream) {
  const ra_status_t st = check_types(dtype, weight_dtype);
  if (st != RA_SUCCESS) return st;
  if (!(eps >= 0.0 && eps < INFINITY) || !shape_ok(rows, cols) || !stride_ok(rows, cols, x_stride) ||
      !stride_ok(rows, cols, y_stride))
    return RA_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RA_SUCCESS;
  const uint64_t es = ra::float_size(dtype), ws = ra::float_size(weight_dtype);
  Buffer in[3] = {{x, extent(rows, cols, x_stride, es), es, true, {}, x_stride * es},
                  {weight, cols * ws, ws, false, {}},
                  {bias, cols * ws, ws, false, {}}};
  Buffer out[3] = {{y, extent(rows, cols, y_stride, es), es, true, {}, y_stride * es},
                   {mean, rows * 4, 4, false, {}},
                   {rstd, rows * 4, 4, false, {}}};
  for (Buffer& b : in)
    if (!sound(b)) return RA_ERR_INVALID_ARG;
  for (Buffer& b : out)
    if (!sound(b)) return RA_ERR_INVALID_ARG;
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i)
      if (shares(out[o], in[i], cols * es) && !(o == 0 && i == 0 && y == x && y_stride == x_stride)) return RA_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (shares(out[o], out[q], cols * es)) return RA_ERR_ALIAS;
  }
  const ra::LnForward a{x, weight, bias, y, mean, rstd, rows, cols, x_stride, y_stride, (float)eps};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == RA_FLOAT32) err = ra::ln_forward_0_0(a, s);
  else if (dtype == RA_FLOAT16) err = weight_dtype == RA_FLOAT32 ? ra::ln_forward_1_0(a, s) : ra::ln_forward_1_1(a, s);
  else err = weight_dtype == RA_FLOAT32 ? ra::ln_forward_2_0(a, s) : ra::ln_forward_2_2(a, s);
  return ra::launched(err);
}

size_t ra_layernorm_workspace(size_t rows, size_t cols) {
  if (!shape_ok(rows, cols)) return 0;
  return (size_t)((rows < kLnMaxParts ? rows : kLnMaxParts) * 2 * cols * 4);
}

ra_status_t ra_layernorm_backward(const void* dy, size_t dy_stride, const void* x, size_t x_stride,
                                  const void* weight, const float* mean, const float* rstd, void* dx,
                                  size_t dx_stride, void* dweight, void* dbias, int accumulate, size_t rows,
                                  size_t cols, ra_dtype_t dtype, ra_dtype_t weight_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const ra_status_t st = check_types(dtype, weight_dtype);
  if (st != RA_SUCCESS) return st;
  if (!shape_ok(rows, cols) || !stride_ok(rows, cols, x_stride) || !stride_ok(rows, cols, dy_stride) ||
      !stride_ok(rows, cols, dx_stride))
    return RA_ERR_INVALID_ARG;
  if (cols == 0) return RA_SUCCESS;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (rows == 0 && (!sums || accumulate)) return RA_SUCCESS;
  const uint64_t es = ra::float_size(dtype), ws = ra::float_size(weight_dtype);
  const uint64_t scratch = sums ? ra_layernorm_workspace(rows, cols) : 0;
  if (workspace_bytes < scratch) return RA_ERR_INVALID_ARG;
  const auto full = [&](size_t stride) { return rows ? extent(rows, cols, stride, es) : 0; };
  Buffer in[5] = {{dy, full(dy_stride), es, rows > 0, {}, dy_stride * es},
                  {x, full(x_stride), es, rows > 0, {}, x_stride * es},
                  {weight, cols * ws, ws, false, {}},
                  {mean, rows * 4, 4, rows > 0, {}},
                  {rstd, rows * 4, 4, rows > 0, {}}};
  Buffer out[4] = {{dx, full(dx_stride), es, rows > 0, {}, dx_stride * es},
                   {dweight, cols * ws, ws, false, {}},
                   {dbias, cols * ws, ws, false, {}},
                   {scratch ? workspace : nullptr, scratch, 16, scratch > 0, {}}};
  for (Buffer& b : in)
    if (!sound(b)) return RA_ERR_INVALID_ARG;
  for (Buffer& b : out)
    if (!sound(b)) return RA_ERR_INVALID_ARG;
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i) {
      const bool same =
          o == 0 && ((i == 0 && dx == dy && dx_stride == dy_stride) || (i == 1 && dx == x && dx_stride == x_stride));
      if (shares(out[o], in[i], cols * es) && !same) return RA_ERR_ALIAS;
    }
    for (int q = 0; q < o; ++q)
      if (shares(out[o], out[q], cols * es)) return RA_ERR_ALIAS;
  }
  ra::LnBackward a{dy, x, weight, mean, rstd, dx, dweight, dbias, static_cast<float*>(workspace), rows, cols,
                   dy_stride, x_stride, dx_stride, accumulate, 0, 0, 1, 0};
  a.parts = (int)(rows < kLnMaxParts ? rows : kLnMaxParts);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == RA_FLOAT32) err = ra::ln_backward_0_0(a, s);
  else if (dtype == RA_FLOAT16) err = weight_dtype == RA_FLOAT32 ? ra::ln_backward_1_0(a, s) : ra::ln_backward_1_1(a, s);
  else err = weight_dtype == RA_FLOAT32 ? ra::ln_backward_2_0(a, s) : ra::ln_backward_2_2(a, s);
  return ra::launched(err);
}

}  // extern "C"
