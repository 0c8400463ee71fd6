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
  uint32_t group;  // threads per row of the register kernel
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
  uint32_t group;   // threads per row of the fused kernel
  uint32_t stages;  // rows a group of it has in shared memory
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

// ---- rows in registers ------------------------------------------------------
// A group of `group` threads (a power of two from 32) takes a row, each thread
// E of its columns: vectors of V elements (16 bytes), or single elements where
// alignment or an odd row length rules vectors out. Thread t's j-th vector is
// the (j group + t)-th of the row, so a warp's accesses are contiguous.
// 16 bytes of DT, or one element, as fp32.
template <int DT, int V>
__device__ __forceinline__ void widen(const uint4& q, float* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == DT_F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        f[2 * k] = p.x, f[2 * k + 1] = p.y;
      } else {
        f[2 * k] = __uint_as_float(w[k] << 16), f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (DT == DT_F16) {
    const __half2 h = __float22half2_rn(make_float2(a, b));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __float22bfloat162_rn(make_float2(a, b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int DT>
__device__ __forceinline__ uint4 narrow(const float* f) {
  if constexpr (DT == DT_F32)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(narrow2<DT>(f[0], f[1]), narrow2<DT>(f[2], f[3]), narrow2<DT>(f[4], f[5]), narrow2<DT>(f[6], f[7]));
}
// V elements at element i of a weight vector, through L1: every row reads them again.
template <int DT, int V>
__device__ __forceinline__ void load_weights(const void* base, uint64_t i, float* f) {
  constexpr int es = Elem<DT>::kSize;
  const char* p = static_cast<const char*>(base) + i * es;
  if constexpr (V == 1) {
    if constexpr (DT == DT_F32) f[0] = __ldg(reinterpret_cast<const float*>(p));
    else f[0] = widen16<DT>(__ldg(reinterpret_cast<const unsigned short*>(p)));
  } else {
    constexpr int per = 16 / es;
#pragma unroll
    for (int k = 0; k < V / per; ++k) widen<DT, per>(__ldg(reinterpret_cast<const uint4*>(p) + k), f + k * per);
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// All threads of a row's group (a named barrier of its own, or the warp).
__device__ __forceinline__ void group_sync(uint32_t g, uint32_t size) {
  if (size == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(size) : "memory");
}
// The sum over a group, in all its threads, in a fixed order. `slots`: one float per warp of the CTA; the
// caller alternates between two sets, so one barrier is enough.
__device__ __forceinline__ float group_sum(float x, uint32_t g, uint32_t size, float* slots) {
  x = warp_sum(x);
  if (size == 32) return x;
  const uint32_t warps = size / 32, first = g * warps;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x / 32] = x;
  group_sync(g, size);
  x = (threadIdx.x & 31) < warps ? slots[first + (threadIdx.x & 31)] : 0.0f;
  return warp_sum(x);
}

constexpr uint32_t kLnMaxThreads = 512;

template <int DT, int WDT, int E, bool VECTOR>
__global__ void __launch_bounds__(kLnMaxThreads) ln_forward_registers(const __grid_constant__ LnForward a) {
  pdl_enter();
  constexpr int es = Elem<DT>::kSize, V = VECTOR ? 16 / es : 1, NV = E / V;
  __shared__ float slots[2][kLnMaxThreads / 32];
  const uint32_t g = threadIdx.x / a.group, t = threadIdx.x - g * a.group;
  const uint64_t row = (uint64_t)blockIdx.x * (blockDim.x / a.group) + g;
  if (row >= a.rows) return;  // a whole group
  const uint32_t cols = (uint32_t)a.cols, step = a.group * V;
  const char* x = static_cast<const char*>(a.x) + row * a.x_stride * es;
  char* y = static_cast<char*>(a.y) + row * a.y_stride * es;
  float f[E];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t c = j * step + t * V;
    if (c < cols) {
      if constexpr (VECTOR) widen<DT, V>(__ldcs(reinterpret_cast<const uint4*>(x + (uint64_t)c * es)), f + j * V);
      else f[j] = ln_load<DT>(x, c);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) f[j * V + k] = 0.0f;
    }
  }
#pragma unroll
  for (int k = 0; k < E; ++k) sum += f[k];
  const float n = (float)cols;
  const float mean = __fdiv_rn(group_sum(sum, g, a.group, slots[0]), n);  // divided: a constant row's mean is exact
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = j * step + t * V < cols;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      f[j * V + k] -= mean;
      if (in) sq = __fmaf_rn(f[j * V + k], f[j * V + k], sq);
    }
  }
  const float var = __fdiv_rn(group_sum(sq, g, a.group, slots[1]), n);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t c = j * step + t * V;
    if (c >= cols) continue;
    float w[V], b[V], out[V];
#pragma unroll
    for (int k = 0; k < V; ++k) w[k] = 1.0f, b[k] = 0.0f;
    if (a.w) load_weights<WDT, V>(a.w, c, w);
    if (a.b) load_weights<WDT, V>(a.b, c, b);
#pragma unroll
    for (int k = 0; k < V; ++k) out[k] = __fmaf_rn(f[j * V + k] * rstd, w[k], b[k]);
    if constexpr (VECTOR) __stcs(reinterpret_cast<uint4*>(y + (uint64_t)c * es), narrow<DT>(out));
    else ln_store<DT>(y, c, out[0]);
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ---- the backward pass in one sweep --------------------------------------------
// One CTA per SM; its groups walk over the rows. The next rows of x and dy are
// on their way into shared memory (cp.async) while a row is worked on, and the
// column sums of dy xhat and dy stay in registers over all the rows of a group:
// x and dy are read once. The CTA folds its groups' sums and writes one partial
// of each; ln_backward_finish adds the partials.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  // copies `bytes` (0 to 16) and fills up with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bytes of one row's buffer in shared memory: single-element rows keep their offset in a 16-byte line.
__host__ __device__ constexpr uint32_t ln_row_bytes(uint32_t cols, uint32_t es, bool vector) {
  return (cols * es + (vector ? 0 : 16) + 15) / 16 * 16;
}

template <int DT, int WDT, int E, bool VECTOR>
__global__ void __launch_bounds__(kLnMaxThreads, 1) ln_backward_fused(const __grid_constant__ LnBackward a) {
  pdl_enter();
  constexpr uint32_t es = Elem<DT>::kSize, V = VECTOR ? 16 / es : 1, NV = E / V;
  extern __shared__ __align__(16) char smem[];
  __shared__ float slots[2][2][kLnMaxThreads / 32];
  const uint32_t cols = (uint32_t)a.cols, size = a.group, groups = kLnMaxThreads / size, stages = a.stages;
  const uint32_t g = threadIdx.x / size, t = threadIdx.x - g * size, step = size * V;
  const uint32_t row_bytes = ln_row_bytes(cols, es, VECTOR);
  float* weights = reinterpret_cast<float*>(smem);
  char* ring = smem + (cols * 4 + 15) / 16 * 16 + (size_t)g * stages * 2 * row_bytes;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  for (uint32_t c = threadIdx.x; c < cols; c += kLnMaxThreads) weights[c] = a.w ? ln_load<WDT>(a.w, c) : 1.0f;
  __syncthreads();

  const char* xs = static_cast<const char*>(a.x);
  const char* dys = static_cast<const char*>(a.dy);
  // few rows spread over the CTAs first, then over their groups
  const uint64_t first = (uint64_t)g * gridDim.x + blockIdx.x, stride = (uint64_t)gridDim.x * groups;
  const char* x_end = xs + ((a.rows - 1) * a.x_stride + cols) * es;
  const char* dy_end = dys + ((a.rows - 1) * a.dy_stride + cols) * es;
  // Copies a row into a buffer. Single-element rows: the 16-byte lines that hold it, none read outside the matrix.
  const auto fetch_row = [&](uint32_t dst, const char* base, const char* end, const char* row) {
    if constexpr (VECTOR) {
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        const uint32_t c = j * step + t * V;
        if (c < cols) cp_async16(dst + c * es, row + (uint64_t)c * es, 16);
      }
    } else {
      const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
      const char* line0 = row - off;
      for (uint32_t k = t; k * 16 < off + cols * es; k += size) {
        const char* line = line0 + k * 16;
        if (line >= base) {
          const uint64_t left = (uint64_t)(end - line);
          cp_async16(dst + k * 16, line, left < 16 ? (uint32_t)left : 16);
        } else {  // the matrix starts inside this line
          for (uint32_t b = off; b < 16 && b < off + cols * es; b += es) {
            const uint32_t bits = ld_elem<DT>(row, (b - off) / es);
            if constexpr (es == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + b), "r"(bits) : "memory");
            else asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + b), "h"((unsigned short)bits) : "memory");
          }
        }
      }
    }
  };
  const auto fetch = [&](uint32_t stage, uint64_t row) {
    if (row < a.rows) {
      fetch_row(ring_at + stage * 2 * row_bytes, xs, x_end, xs + row * a.x_stride * es);
      fetch_row(ring_at + (stage * 2 + 1) * row_bytes, dys, dy_end, dys + row * a.dy_stride * es);
    }
    cp_async_commit();
  };
  float dw[E], db[E];
#pragma unroll
  for (int k = 0; k < E; ++k) dw[k] = db[k] = 0.0f;
  const float inv_n = 1.0f / (float)cols;
  for (uint32_t s = 0; s + 1 < stages; ++s) fetch(s, first + s * stride);
  float mean = 0.0f, rstd = 0.0f;
  if (first < a.rows) mean = __ldg(a.mean + first), rstd = __ldg(a.rstd + first);
  uint32_t stage = 0, parity = 0;
  for (uint64_t row = first; row < a.rows; row += stride) {
    if (stages == 2) cp_async_wait<0>();
    else if (stages == 3) cp_async_wait<1>();
    else cp_async_wait<2>();
    if constexpr (!VECTOR) group_sync(g, size);  // the row was copied by all; and all are done with the one before
    fetch(stage == 0 ? stages - 1 : stage - 1, row + (stages - 1) * stride);
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (row + stride < a.rows) next_mean = __ldg(a.mean + row + stride), next_rstd = __ldg(a.rstd + row + stride);

    const char* sx = ring + stage * 2 * row_bytes;
    const char* sdy = sx + row_bytes;
    if constexpr (!VECTOR) {
      sx += reinterpret_cast<uintptr_t>(xs + row * a.x_stride * es) & 15;
      sdy += reinterpret_cast<uintptr_t>(dys + row * a.dy_stride * es) & 15;
    }
    const auto load = [&](uint32_t c, float* x, float* dy, float* w) {
      if constexpr (VECTOR) {
        widen<DT, V>(*reinterpret_cast<const uint4*>(sx + c * es), x);
        widen<DT, V>(*reinterpret_cast<const uint4*>(sdy + c * es), dy);
#pragma unroll
        for (uint32_t k = 0; k < V; k += 4) {
          const float4 q = *reinterpret_cast<const float4*>(weights + c + k);
          w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
        }
      } else {
        if constexpr (DT == DT_F32) {
          x[0] = *reinterpret_cast<const float*>(sx + c * es), dy[0] = *reinterpret_cast<const float*>(sdy + c * es);
        } else {
          x[0] = widen16<DT>(*reinterpret_cast<const unsigned short*>(sx + c * es));
          dy[0] = widen16<DT>(*reinterpret_cast<const unsigned short*>(sdy + c * es));
        }
        w[0] = weights[c];
      }
    };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      const uint32_t c = j * step + t * V;
      if (c >= cols) continue;
      float x[V], dy[V], w[V];
      load(c, x, dy, w);
#pragma unroll
      for (uint32_t k = 0; k < V; ++k) {
        const float h = (x[k] - mean) * rstd, p = dy[k] * w[k];
        s1 += p;
        s2 = __fmaf_rn(p, h, s2);
        dw[j * V + k] = __fmaf_rn(dy[k], h, dw[j * V + k]);
        db[j * V + k] += dy[k];
      }
    }
    // both sums in one exchange
    s1 = warp_sum(s1), s2 = warp_sum(s2);
    if (size > 32) {
      const uint32_t warps = size / 32, lane = threadIdx.x & 31;
      if (lane == 0) slots[parity][0][threadIdx.x / 32] = s1, slots[parity][1][threadIdx.x / 32] = s2;
      group_sync(g, size);
      s1 = warp_sum(lane < warps ? slots[parity][0][g * warps + lane] : 0.0f);
      s2 = warp_sum(lane < warps ? slots[parity][1][g * warps + lane] : 0.0f);
      parity ^= 1;
    }
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
    char* dx = static_cast<char*>(a.dx) + row * a.dx_stride * es;
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      const uint32_t c = j * step + t * V;
      if (c >= cols) continue;
      float x[V], dy[V], w[V], out[V];
      load(c, x, dy, w);
#pragma unroll
      for (uint32_t k = 0; k < V; ++k) {
        const float h = (x[k] - mean) * rstd;
        out[k] = rstd * (__fmaf_rn(dy[k], w[k], -c1) - h * c2);
      }
      if constexpr (VECTOR) __stcs(reinterpret_cast<uint4*>(dx + (uint64_t)c * es), narrow<DT>(out));
      else ln_store<DT>(dx, c, out[0]);
    }
    mean = next_mean, rstd = next_rstd;
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  if (a.dw == nullptr && a.db == nullptr) return;
  // fold the groups: every group's sums side by side in shared memory, then column by column
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
    const uint32_t c = j * step + t * V;
    if (c >= cols) continue;
#pragma unroll
    for (uint32_t k = 0; k < V; ++k) {
      sums[(g * 2) * cols + c + k] = dw[j * V + k];
      sums[(g * 2 + 1) * cols + c + k] = db[j * V + k];
    }
  }
  __syncthreads();
  float* part = a.part + (uint64_t)blockIdx.x * 2 * cols;
  for (uint32_t c = threadIdx.x; c < 2 * cols; c += kLnMaxThreads) {
    float s = sums[c];
    for (uint32_t k = 1; k < groups; ++k) s += sums[k * 2 * cols + c];
    part[c] = s;
  }
}

// ---- rows of any length ------------------------------------------------------------
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
