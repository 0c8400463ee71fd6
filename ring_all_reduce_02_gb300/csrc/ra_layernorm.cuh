// Layer norm over the rows of a matrix, forward and backward.
//
// Forward: mean, then the centred sum of squares (two sums over the row: the
// difference of raw moments would cancel where |mean| is large against the
// deviation), then y = (x - mean) rstd w + b.
// Backward, with xhat = (x - mean) rstd and a = dy w, both sums over the row:
//   dx = rstd (a - sum(a)/n - xhat sum(a xhat)/n),
// and over the rows: dw = sum dy xhat, db = sum dy.
#pragma once

#include "ra_kernels.cuh"
#include "ra_ops.cuh"

namespace ra {

struct LnForward {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  uint64_t rows, cols, x_stride, y_stride;
  float eps;
};

struct LnBackward {
  const void* dy;
  const void* x;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dw;
  void* db;
  float* part;  // [parts][2][cols]: partial sums of dw and db
  uint64_t rows, cols, dy_stride, x_stride, dx_stride;
  int accumulate;
  int parts;
};

template <int DT>
__device__ __forceinline__ float ln_load(const void* base, uint64_t i) {
  if constexpr (DT == DT_F32) return __uint_as_float(ld_elem<DT>(base, i));
  else return widen16<DT>(ld_elem<DT>(base, i));
}
template <int DT>
__device__ __forceinline__ void ln_store(void* base, uint64_t i, float x) {
  if constexpr (DT == DT_F32) st_elem<DT>(base, i, __float_as_uint(x));
  else st_elem<DT>(base, i, round16<DT>(x));
}

// The sum over the CTA, in every thread; a fixed tree. `smem`: 33 floats, free again after the next barrier.
template <int THREADS>
__device__ __forceinline__ float cta_sum_all(float x, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x / 32] = x;
  __syncthreads();
  x = (threadIdx.x & 31) < THREADS / 32 ? smem[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

constexpr int kLnThreads = 256;

template <int DT, int WDT>
__global__ void __launch_bounds__(kLnThreads) ln_forward_rows(const __grid_constant__ LnForward a) {
  pdl_enter();
  __shared__ float smem[33];
  constexpr int es = Elem<DT>::kSize;
  const float n = (float)a.cols;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + row * a.x_stride * es;
    char* y = static_cast<char*>(a.y) + row * a.y_stride * es;
    float sum = 0.0f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) sum += ln_load<DT>(x, i);
    const float mean = __fdiv_rn(cta_sum_all<kLnThreads>(sum, smem), n);  // divided: a constant row's mean is exact
    float sq = 0.0f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) {
      const float d = ln_load<DT>(x, i) - mean;
      sq = __fmaf_rn(d, d, sq);
    }
    const float var = __fdiv_rn(cta_sum_all<kLnThreads>(sq, smem), n);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) {
      const float w = a.w ? ln_load<WDT>(a.w, i) : 1.0f, b = a.b ? ln_load<WDT>(a.b, i) : 0.0f;
      ln_store<DT>(y, i, __fmaf_rn((ln_load<DT>(x, i) - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kLnThreads) ln_backward_rows(const __grid_constant__ LnBackward a) {
  pdl_enter();
  __shared__ float smem[33];
  constexpr int es = Elem<DT>::kSize;
  const float inv_n = 1.0f / (float)a.cols;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + row * a.x_stride * es;
    const char* dy = static_cast<const char*>(a.dy) + row * a.dy_stride * es;
    char* dx = static_cast<char*>(a.dx) + row * a.dx_stride * es;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) {
      const float w = a.w ? ln_load<WDT>(a.w, i) : 1.0f;
      const float g = ln_load<DT>(dy, i) * w, h = (ln_load<DT>(x, i) - mean) * rstd;
      s1 += g;
      s2 = __fmaf_rn(g, h, s2);
    }
    s1 = cta_sum_all<kLnThreads>(s1, smem) * inv_n;
    s2 = cta_sum_all<kLnThreads>(s2, smem) * inv_n;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) {
      const float w = a.w ? ln_load<WDT>(a.w, i) : 1.0f;
      const float g = ln_load<DT>(dy, i) * w, h = (ln_load<DT>(x, i) - mean) * rstd;
      ln_store<DT>(dx, i, rstd * (g - s1 - h * s2));
    }
  }
}

// Partial sums over a share of the rows: CTA (x, y) takes 32 columns and part y's rows.
template <int DT>
__global__ void __launch_bounds__(kLnThreads) ln_backward_columns(const __grid_constant__ LnBackward a) {
  pdl_enter();
  __shared__ float sw[kLnThreads / 32][33], sb[kLnThreads / 32][33];
  constexpr int es = Elem<DT>::kSize;
  const uint32_t lane = threadIdx.x & 31, wid = threadIdx.x / 32;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  float dw = 0.0f, db = 0.0f;
  if (c < a.cols) {
    for (uint64_t row = (uint64_t)blockIdx.y * (kLnThreads / 32) + wid; row < a.rows;
         row += (uint64_t)a.parts * (kLnThreads / 32)) {
      const float g = ln_load<DT>(static_cast<const char*>(a.dy) + row * a.dy_stride * es, c);
      const float h = (ln_load<DT>(static_cast<const char*>(a.x) + row * a.x_stride * es, c) - a.mean[row]) * a.rstd[row];
      dw = __fmaf_rn(g, h, dw);
      db += g;
    }
  }
  sw[wid][lane] = dw, sb[wid][lane] = db;
  __syncthreads();
  if (wid == 0 && c < a.cols) {
    for (int k = 1; k < kLnThreads / 32; ++k) dw += sw[k][lane], db += sb[k][lane];
    a.part[(uint64_t)blockIdx.y * 2 * a.cols + c] = dw;
    a.part[((uint64_t)blockIdx.y * 2 + 1) * a.cols + c] = db;
  }
}

// The sums of the partials: CTA x takes 32 columns.
template <int WDT>
__global__ void __launch_bounds__(kLnThreads) ln_backward_finish(const __grid_constant__ LnBackward a) {
  pdl_enter();
  __shared__ float sw[kLnThreads / 32][33], sb[kLnThreads / 32][33];
  const uint32_t lane = threadIdx.x & 31, wid = threadIdx.x / 32;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  float dw = 0.0f, db = 0.0f;
  if (c < a.cols) {
    for (int p = wid; p < a.parts; p += kLnThreads / 32) {
      dw += a.part[(uint64_t)p * 2 * a.cols + c];
      db += a.part[((uint64_t)p * 2 + 1) * a.cols + c];
    }
  }
  sw[wid][lane] = dw, sb[wid][lane] = db;
  __syncthreads();
  if (wid == 0 && c < a.cols) {
    for (int k = 1; k < kLnThreads / 32; ++k) dw += sw[k][lane], db += sb[k][lane];
    if (a.dw) ln_store<WDT>(a.dw, c, a.accumulate ? ln_load<WDT>(a.dw, c) + dw : dw);
    if (a.db) ln_store<WDT>(a.db, c, a.accumulate ? ln_load<WDT>(a.db, c) + db : db);
  }
}

}  // namespace ra
