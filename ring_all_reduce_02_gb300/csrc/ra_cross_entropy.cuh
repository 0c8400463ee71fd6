// Softmax cross entropy from the hidden states h [T, D] and the head's weight w [V, D], in 16 bits.
//
//   forward    logit = h w^T, lse = log sum exp(logit), loss = lse - logit[target]
//   backward   g = dloss (exp(logit - lse) - onehot),  dh = g w,  dw = g^T h
//
// Rows without a loss are left out: a first kernel numbers the others, a second copies their hidden states side by side
// (which also makes them whole 16-byte lines), and every product runs over the rows that count alone. The logits are
// not stored: the forward pass folds every tile of them into a partial maximum and sum per row, which a last kernel
// joins; the backward pass computes them again, a piece of the vocabulary at a time, and stores that piece of g.
#pragma once

#include <cuda_runtime.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"
#include "ra_tokens.cuh"

namespace ra {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct CeHeader {
  int32_t rows;  // that count
  int32_t pad;
  float scale;   // the largest finite |dloss| (1 if that is 0)
};

// Everything that the kernels need.
struct CeArgs {
  const void *hidden, *weight;  // as given
  const void *h, *w;            // hidden's copy; the weight, or its copy
  uint64_t hidden_stride, weight_stride, w_stride;
  Indices targets;
  int64_t ignore;
  uint64_t rows, cols, vocab, rows_pad, cols_pad, slots, piece;
  CeHeader* head;
  int32_t *index, *where, *target;  // row of a counted row; counted row of a row or -1; its target or -1 (no number of the vocabulary)
  float *lse_kept, *dloss_kept;     // backward: of the counted rows
  float* logit;                     // forward: the target's logit of a counted row
  float2* partial;                  // forward: [rows_pad][slots]
  void* g;                          // backward: [rows_pad][piece]
  float* dh;                        // backward: [rows_pad][cols_pad]
  float *loss, *lse;                // forward: outputs; backward: lse is an input
  const float* dloss;
  void *dhidden, *dweight;
  uint64_t dhidden_stride, dweight_stride;
  int accumulate;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---- rows that count ---------------------------------------------------------------

constexpr int kCeRowsThreads = 1024;

// One CTA: numbers the rows that count in their order.
template <bool BACKWARD>
__global__ void __launch_bounds__(kCeRowsThreads) ce_rows_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  __shared__ int32_t sums[32];
  __shared__ float tops[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int32_t before = 0;
  float top = 0.0f;
  for (uint64_t t0 = 0; t0 < a.rows; t0 += kCeRowsThreads) {
    const uint64_t t = t0 + threadIdx.x;
    const int64_t v = t < a.rows ? load_index(a.targets, t) : a.ignore;
    const bool counts = v != a.ignore;
    const uint32_t votes = __ballot_sync(0xffffffffu, counts);
    if (lane == 0) sums[warp] = __popc(votes);
    __syncthreads();
    int32_t sum = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int32_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    const int32_t all = __shfl_sync(0xffffffffu, sum, 31);
    const int32_t mine = before + (warp ? __shfl_sync(0xffffffffu, sum, warp - 1) : 0) + __popc(votes & ((1u << lane) - 1));
    if (counts) {
      a.index[mine] = (int32_t)t;
      a.target[mine] = v >= 0 && v < (int64_t)a.vocab ? (int32_t)v : -1;
      if constexpr (BACKWARD) {
        const float d = a.dloss ? a.dloss[t] : 1.0f;
        a.lse_kept[mine] = a.lse[t];
        a.dloss_kept[mine] = d;
        if (fabsf(d) < __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(d));
      }
    } else if (!BACKWARD && t < a.rows) {
      a.loss[t] = 0.0f;
      a.lse[t] = 0.0f;
    }
    if (t < a.rows) a.where[t] = counts ? mine : -1;
    before += all;
    __syncthreads();
  }
  if constexpr (BACKWARD) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (threadIdx.x == 0) {
    a.head->rows = before;
    a.head->scale = top > 0.0f ? top : 1.0f;
  }
}

// The counted rows' hidden states side by side, zeros behind them.
__global__ void __launch_bounds__(256) ce_hidden_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, up = (rows + 255) / 256 * 256;
  for (uint64_t i = blockIdx.x; i < up; i += gridDim.x) {
    uint16_t* to = static_cast<uint16_t*>(const_cast<void*>(a.h)) + i * a.cols_pad;
    const uint16_t* from = i < rows ? static_cast<const uint16_t*>(a.hidden) + (uint64_t)a.index[i] * a.hidden_stride : nullptr;
    for (uint64_t c = threadIdx.x; c < a.cols_pad; c += 256) to[c] = from && c < a.cols ? from[c] : (uint16_t)0;
  }
}

// The weight in rows of whole 16-byte lines.
__global__ void __launch_bounds__(256) ce_weight_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  for (uint64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
    uint16_t* to = static_cast<uint16_t*>(const_cast<void*>(a.w)) + v * a.w_stride;
    const uint16_t* from = static_cast<const uint16_t*>(a.weight) + v * a.weight_stride;
    for (uint64_t c = threadIdx.x; c < a.cols_pad; c += 256) to[c] = c < a.cols ? from[c] : (uint16_t)0;
  }
}

// ---- products ------------------------------------------------------------------------

// A matrix read as [m][k], wherever its elements lie.
struct CeOperand {
  const void* p;
  uint64_t m_stride, k_stride, m_size, k_size;
};
template <int DT>
__device__ __forceinline__ float ce_element(const CeOperand& o, uint64_t m, uint64_t k) {
  if (m >= o.m_size || k >= o.k_size) return 0.0f;
  return widen16<DT>(static_cast<const uint16_t*>(o.p)[m * o.m_stride + k * o.k_stride]);
}

// 64 x 64 elements of A B^T by 256 threads, 4 x 4 each: thread t has rows 4 (t / 16) and columns 4 (t % 16) on.
template <int DT>
__device__ __forceinline__ void ce_tile(const CeOperand& a, const CeOperand& b, uint64_t m0, uint64_t n0, float acc[4][4]) {
  __shared__ float as[16][65], bs[16][65];
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (uint64_t k0 = 0; k0 < a.k_size; k0 += 16) {
    for (int e = threadIdx.x; e < 1024; e += 256) {
      as[e % 16][e / 16] = ce_element<DT>(a, m0 + e / 16, k0 + e % 16);
      bs[e % 16][e / 16] = ce_element<DT>(b, n0 + e / 16, k0 + e % 16);
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(as[k][4 * tm + i], bs[k][4 * tn + j], acc[i][j]);
    __syncthreads();
  }
}

// The forward pass's tiles: the maximum and the sum of each row's 64 logits, and the target's logit.
template <int DT>
__global__ void __launch_bounds__(256) ce_logits_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, m0 = (uint64_t)blockIdx.y * 64, n0 = (uint64_t)blockIdx.x * 64;
  if (m0 >= rows) return;
  float acc[4][4];
  ce_tile<DT>({a.h, a.cols_pad, 1, rows, a.cols}, {a.w, a.w_stride, 1, a.vocab, a.cols}, m0, n0, acc);
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  const float low = __int_as_float(0xff800000);
  for (int i = 0; i < 4; ++i) {
    const uint64_t m = m0 + 4 * tm + i;
    float top = low, sum = 0.0f;
    for (int j = 0; j < 4; ++j)
      if (n0 + 4 * tn + j < a.vocab) top = fmaxf(top, acc[i][j]);
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == low ? 0.0f : top;  // a row of -inf alone has the sum 0
    for (int j = 0; j < 4; ++j)
      if (n0 + 4 * tn + j < a.vocab) sum += exp2_approx(__fmul_rn(acc[i][j] - base, kLog2e));
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (m >= rows) continue;
    if (tn == 0) a.partial[m * a.slots + blockIdx.x] = make_float2(top, sum);
    const int64_t at = (int64_t)a.target[m] - (int64_t)(n0 + 4 * tn);
    for (int j = 0; j < 4; ++j)
      if (at == j) a.logit[m] = acc[i][j];
  }
}

// Joins a row's partial sums: a warp per counted row.
__global__ void __launch_bounds__(256) ce_join_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const uint64_t i = (uint64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (i >= (uint64_t)a.head->rows) return;
  const int lane = threadIdx.x & 31;
  const float low = __int_as_float(0xff800000);
  float top = low, sum = 0.0f;
  for (uint64_t s = lane; s < a.slots; s += 32) {
    const float2 p = a.partial[i * a.slots + s];
    const float both = fmaxf(top, p.x), base = both == low ? 0.0f : both;
    sum = sum * exp2_approx((top - base) * kLog2e) + p.y * exp2_approx((p.x - base) * kLog2e);
    top = both;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, top, o), osum = __shfl_xor_sync(0xffffffffu, sum, o);
    const float both = fmaxf(top, other), base = both == low ? 0.0f : both;
    sum = sum * exp2_approx((top - base) * kLog2e) + osum * exp2_approx((other - base) * kLog2e);
    top = both;
  }
  if (lane == 0) {
    const bool there = a.target[i] >= 0;
    const float nan = __int_as_float(0x7fffffff);
    const float lse = there ? top + logf(sum) : nan;
    const uint64_t t = (uint64_t)a.index[i];
    a.lse[t] = lse;
    a.loss[t] = there ? lse - a.logit[i] : nan;
  }
}

// A piece of g, from the logits computed again; rows behind the counted ones are zero.
template <int DT>
__global__ void __launch_bounds__(256) ce_g_kernel(const __grid_constant__ CeArgs a, uint64_t v0) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, m0 = (uint64_t)blockIdx.y * 64, n0 = v0 + (uint64_t)blockIdx.x * 64;
  if (m0 >= (rows + 255) / 256 * 256) return;
  float acc[4][4];
  ce_tile<DT>({a.h, a.cols_pad, 1, rows, a.cols}, {a.w, a.w_stride, 1, a.vocab, a.cols}, m0, n0, acc);
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i) {
    const uint64_t m = m0 + 4 * tm + i;
    const bool counts = m < rows;
    const float lse = counts ? a.lse_kept[m] : 0.0f;
    const int32_t target = counts ? a.target[m] : -1;
    float d = counts ? __fdiv_rn(a.dloss_kept[m], a.head->scale) : 0.0f;
    if (counts && target < 0) d = __int_as_float(0x7fffffff);
    for (int j = 0; j < 4; ++j) {
      const uint64_t v = n0 + 4 * tn + j;
      float g = 0.0f;
      if (counts && v < a.vocab) {
        g = exp2_approx(__fmul_rn(acc[i][j] - lse, kLog2e));
        if ((int64_t)v == target) g -= 1.0f;
        g *= d;
      }
      static_cast<uint16_t*>(a.g)[m * a.piece + (v - v0)] = (uint16_t)round16<DT>(g * (DT == DT_F16 ? 16384.0f : 1.0f));
    }
  }
}

// dh += g w over a piece.
template <int DT>
__global__ void __launch_bounds__(256) ce_dhidden_kernel(const __grid_constant__ CeArgs a, uint64_t v0, uint64_t width) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, m0 = (uint64_t)blockIdx.y * 64, n0 = (uint64_t)blockIdx.x * 64;
  if (m0 >= rows) return;
  float acc[4][4];
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + v0 * a.w_stride;
  ce_tile<DT>({a.g, a.piece, 1, rows, width}, {w, 1, a.w_stride, a.cols, width}, m0, n0, acc);
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const uint64_t m = m0 + 4 * tm + i, c = n0 + 4 * tn + j;
      if (m >= rows || c >= a.cols) continue;
      float* at = a.dh + m * a.cols_pad + c;
      *at = v0 ? *at + acc[i][j] : acc[i][j];
    }
}

template <int DT>
__device__ __forceinline__ void ce_store(void* p, uint64_t i, float f) {
  if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = f;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)round16<DT>(f);
}
template <int DT>
__device__ __forceinline__ float ce_load(const void* p, uint64_t i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return widen16<DT>(static_cast<const uint16_t*>(p)[i]);
}
// What g is multiplied by where it is used.
template <int DT>
__device__ __forceinline__ float ce_unscale(const CeArgs& a) { return a.head->scale * (DT == DT_F16 ? 1.0f / 16384.0f : 1.0f); }

// dw (+)= g^T h over a piece.
template <int DT, int WDT>
__global__ void __launch_bounds__(256) ce_dweight_kernel(const __grid_constant__ CeArgs a, uint64_t v0, uint64_t width) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, m0 = (uint64_t)blockIdx.y * 64, n0 = (uint64_t)blockIdx.x * 64;
  float acc[4][4];
  ce_tile<DT>({a.g, 1, a.piece, width, rows}, {a.h, 1, a.cols_pad, a.cols, rows}, m0, n0, acc);
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const uint64_t m = m0 + 4 * tm + i, c = n0 + 4 * tn + j;
      if (m >= width || c >= a.cols) continue;
      const uint64_t at = (v0 + m) * a.dweight_stride + c;
      float x = acc[i][j] * ce_unscale<DT>(a);
      if (a.accumulate) x += ce_load<WDT>(a.dweight, at);
      ce_store<WDT>(a.dweight, at, x);
    }
}

// dh into the rows it belongs to, zeros into those that do not count.
template <int DT>
__global__ void __launch_bounds__(256) ce_finish_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const int32_t i = a.where[t];
    for (uint64_t c = threadIdx.x; c < a.cols; c += 256)
      ce_store<DT>(a.dhidden, t * a.dhidden_stride + c, i < 0 ? 0.0f : a.dh[(uint64_t)i * a.cols_pad + c] * ce_unscale<DT>(a));
  }
}

}  // namespace ra
