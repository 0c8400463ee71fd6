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
#include "ra_pairs.cuh"

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

// Partial sums of the weight's gradient, at most: one per SM. A multiple of 8, see ln_backward_fused.
constexpr uint64_t kLnMaxParts = 152;
constexpr uint32_t kLnMaxSplit = 4;  // CTAs that share a row

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
  uint32_t split;   // CTAs per row of it
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

// 16 bytes of DT as pairs of fp32, and back.
template <int DT>
__device__ __forceinline__ void widen(const uint4& q, F2* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (DT == DT_F32) {
    f[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
    f[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == DT_F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        f[k] = pair(p.x, p.y);
      } else {
        f[k] = pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ uint32_t narrow2(F2 p) {
  float a, b;
  split(p, a, b);
  if constexpr (DT == DT_F16) {
    const __half2 h = __float22half2_rn(make_float2(a, b));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __float22bfloat162_rn(make_float2(a, b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int DT>
__device__ __forceinline__ uint4 narrow(const F2* f) {
  if constexpr (DT == DT_F32) {
    float a, b, c, d;
    split(f[0], a, b), split(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  } else {
    return make_uint4(narrow2<DT>(f[0]), narrow2<DT>(f[1]), narrow2<DT>(f[2]), narrow2<DT>(f[3]));
  }
}
// One weight; other CTAs read it too.
template <int DT>
__device__ __forceinline__ float weight_at(const void* base, uint32_t i) {
  if constexpr (DT == DT_F32) return __ldg(static_cast<const float*>(base) + i);
  else return widen16<DT>(__ldg(static_cast<const unsigned short*>(base) + i));
}
// Where element i of a row's lines has its weight in shared memory: four of a line's values stand together, a
// line's second four `half` floats on, so that a warp's 16-byte reads touch every bank equally often (a thread's
// eight in a row cost two passes: 13% of 6001 x 4095 fp16; backward, 8% of 4096 x 12288 bf16).
template <uint32_t V>
__device__ __forceinline__ uint32_t weight_slot(uint32_t i, uint32_t half) {
  return V == 4 ? i : (i & 4 ? half : 0) + i / 8 * 4 + (i & 3);
}

// V weights from element i, through L1: every row reads them again.
template <int DT, int V>
__device__ __forceinline__ void load_weights(const void* base, uint32_t i, F2* f) {
  constexpr int es = Elem<DT>::kSize, per = 16 / es;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + (uint64_t)i * es);
#pragma unroll
  for (int k = 0; k < V / per; ++k) widen<DT>(__ldg(p + k), f + k * (per / 2));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The sum over the whole CTA of `warps` (up to 16) warps, in all its threads, in a fixed order. `slots`: 16 floats,
// 16-byte aligned; two calls in a row need two sets. A second round of shuffles for more than 4 warps cost 2% to 4%.
__device__ __forceinline__ float cta_sum_registers(float v, float* slots, uint32_t warps) {
  v = warp_sum(v);
  const uint32_t t = threadIdx.x;
  if ((t & 31) == 0) slots[t / 32] = v;
  if (t >= warps && t < (warps + 3) / 4 * 4) slots[t] = 0.0f;
  __syncthreads();
  const float4* at = reinterpret_cast<const float4*>(slots);
  float4 q = at[0];
#pragma unroll
  for (uint32_t k = 1; k < 4; ++k) {
    if (k * 4 >= warps) break;
    const float4 r = at[k];
    q.x += r.x, q.y += r.y, q.z += r.z, q.w += r.w;
  }
  return (q.x + q.y) + (q.z + q.w);
}

constexpr uint32_t kLnMaxThreads = 512;
constexpr uint32_t kLnWarpThreads = 128;  // of a CTA with a row to each warp

// A row's mean from its sum. The product with 1 / n is mended by its remainder, so that a quotient that fp32 holds
// comes out exactly; an infinite sum stays as it is. Three divisions and a square root a row, rounded as IEEE has
// them, cost 4% to 8% of the kernels below.
__device__ __forceinline__ float row_mean(float sum, float n, float inv_n) {
  const float q = sum * inv_n, r = __fmaf_rn(__fmaf_rn(-q, n, sum), inv_n, q);
  return fabsf(q) < INFINITY ? r : q;
}

// A constant row's mean has to be its value: an ulp of a large mean times 1 / deviation = 1 / sqrt(eps) is not small.
// The sum of n equal values of s significant bits is exact in fp32 up to 2^(24 - s) of them. Rows of fp32, and of fp16
// above 8192 columns, can be longer, so there the mean of the deviations from the first mean is added to it: of a
// constant row these are a few ulp, their sum is as good as exact, and the second deviations are zero. bf16 has 8
// bits: exact up to 65,536 columns, which only ln_forward_rows passes. The third exchange costs nothing where HBM
// bounds the row (8192 x 4096 fp32 41.4 -> 41.8 us, 6001 x 4095 fp32 39.6 -> 39.7), up to 15% elsewhere (2047 x 1537
// fp32 7.6 -> 8.3, 2048 x 16384 fp16 28.3 -> 31.4); ln_forward_rows reads the row once more, 9% to 24% for fp32. Sums of
// deviations and squares in one exchange, the variance mended by the difference of the means and summed again where
// that cancels, took 3% to 5% less for fp16 and up to 35% more for odd rows of fp32.
template <int DT>
__host__ __device__ __forceinline__ bool second_mean(uint64_t cols) {
  return DT == DT_F32 || cols > (DT == DT_F16 ? 8192 : 65536);
}
// What to add to a mean, from the mean of the deviations from it: nothing where the row is not finite.
__device__ __forceinline__ float mean_rest(float rest) { return fabsf(rest) < INFINITY ? rest : 0.0f; }

// ---- forward, rows in registers ---------------------------------------------------
// A group of threads takes a row, each of them E of its columns in vectors of
// 16 bytes: thread t's j-th vector is the (j group + t)-th of the row. WARP: a
// row to each warp of a CTA; otherwise the CTA is one row's group (named
// barriers for several groups would hold 16 of an SM's 64 barriers per CTA and
// so allow only 4 CTAs on it).
//
// Measured (back to back, inputs larger than L2): 8192 x 1024 bf16 7.1 us (floor
// 4.9), 8192 x 4096 bf16 23.7 us (83% of the copy bandwidth), 4096 x 8192 fp32
// 41.9 us (94%), 32768 x 8192 bf16 173 us (91%). Short launches spend 2 us on their
// start; at 8192 x 1024 the warps wait for their rows (long_scoreboard) at 52% of
// the issue slots, 16 instructions an element.
template <int DT, int WDT, int E, bool WARP, bool SECOND>
__global__ void __launch_bounds__(WARP ? kLnWarpThreads : kLnMaxThreads) ln_forward_registers(const __grid_constant__ LnForward a) {
  pdl_enter();
  constexpr int es = Elem<DT>::kSize, V = 16 / es, NV = E / V, H = V / 2;
  __shared__ __align__(16) float slots[SECOND ? 3 : 2][kLnMaxThreads / 32];
  const uint32_t group = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const uint64_t row = WARP ? (uint64_t)blockIdx.x * (kLnWarpThreads / 32) + threadIdx.x / 32 : blockIdx.x;
  if (row >= a.rows) return;  // a whole group
  const uint32_t cols = (uint32_t)a.cols, step = group * V;
  const auto group_sum = [&](float v, float* s) { return WARP ? warp_sum(v) : cta_sum_registers(v, s, group / 32); };
  const char* x = static_cast<const char*>(a.x) + row * a.x_stride * es;
  char* y = static_cast<char*>(a.y) + row * a.y_stride * es;
  uint4 q[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t c = j * step + t * V;
    q[j] = c < cols ? __ldcs(reinterpret_cast<const uint4*>(x + c * es)) : make_uint4(0, 0, 0, 0);
  }
  F2 f[E / 2], sum = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    widen<DT>(q[j], f + j * H);
#pragma unroll
    for (int k = 0; k < H; ++k) sum = add2(sum, f[j * H + k]);
  }
  const float n = (float)cols, inv_n = __frcp_rn(n);
  float mean = row_mean(group_sum(fold2(sum), slots[0]), n, inv_n);
  if constexpr (SECOND) {
    const F2 minus = twice(-mean);
    F2 rest = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = j * step + t * V < cols;
#pragma unroll
      for (int k = 0; k < H; ++k)
        if (in) rest = add2(rest, add2(f[j * H + k], minus));
    }
    mean += mean_rest(row_mean(group_sum(fold2(rest), slots[2]), n, inv_n));
  }
  const F2 minus = twice(-mean);
  F2 sq = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = j * step + t * V < cols;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      F2& d = f[j * H + k];
      d = add2(d, minus);
      if (in) sq = fma2(d, d, sq);
    }
  }
  const float var = group_sum(fold2(sq), slots[1]) * inv_n;
  const float rstd = rsqrtf(var + a.eps);
  const F2 rstd2 = twice(rstd);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t c = j * step + t * V;
    if (c >= cols) continue;
    F2 w[H], b[H];
    if (a.w) {
      load_weights<WDT, V>(a.w, c, w);
    } else {
#pragma unroll
      for (int k = 0; k < H; ++k) w[k] = pair(1.0f, 1.0f);
    }
    if (a.b) {
      load_weights<WDT, V>(a.b, c, b);
    } else {
#pragma unroll
      for (int k = 0; k < H; ++k) b[k] = 0;
    }
#pragma unroll
    for (int k = 0; k < H; ++k) w[k] = fma2(mul2(f[j * H + k], rstd2), w[k], b[k]);
    __stcs(reinterpret_cast<uint4*>(y + c * es), narrow<DT>(w));
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ---- rows off the 16-byte grid ---------------------------------------------------------
// A row of an odd length starts somewhere inside a 16-byte line. Its lines are
// read and written whole all the same: a thread's k-th line holds the row's
// elements V k - phase .. V k - phase + V - 1, and what lies outside the row is
// masked. A CTA takes rows that are a multiple of 8 apart, so that all of them
// have one phase, and keeps the weights in shared memory shifted to it.
__device__ __forceinline__ uint32_t line_phase(const void* p, uint32_t es) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u) / es;
}

// Line `at` of the matrix [base, end), element by element where it is not all inside it.
template <int DT>
__device__ __forceinline__ uint4 load_line(const char* at, const char* base, const char* end) {
  if (at >= base && at + 16 <= end) return __ldcs(reinterpret_cast<const uint4*>(at));
  constexpr uint32_t es = Elem<DT>::kSize;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (uint32_t k = 0; k < 16 / es; ++k) {
    const char* p = at + k * es;
    if (p >= base && p < end) w[k * es / 4] |= ld_elem<DT>(p, 0) << (k * es % 4 * 8);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The first `from` and all from `to` on of a line's V values set to zero.
template <uint32_t V>
__device__ __forceinline__ void mask_line(F2* f, int from, int to) {
#pragma unroll
  for (int k = 0; k < (int)V / 2; ++k) {
    float u, v;
    split(f[k], u, v);
    f[k] = pair(2 * k >= from && 2 * k < to ? u : 0.0f, 2 * k + 1 >= from && 2 * k + 1 < to ? v : 0.0f);
  }
}
// Values [from, to) of a line, one by one.
template <int DT>
__device__ __forceinline__ void store_part(char* at, const uint4& q, int from, int to) {
  constexpr uint32_t es = Elem<DT>::kSize;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < (int)(16 / es); ++k)
    if (k >= from && k < to) st_elem<DT>(at, k, es == 4 ? w[k] : (w[k / 2] >> (k % 2 * 16)) & 0xffffu);
}

// Persistent CTAs, one row at a time; the next row's lines are read while a row is worked on. The grid is a
// multiple of 8 (or has a CTA for every row). 6001 x 4095 fp16: 22.8 us (floor 14.5; element by element 75), 2047 x
// 1537 fp32: 8.2 us (3.7). The chain of weights from shared memory and the two or three exchanges of a row on 24 to 32
// resident warps bound it: 2 to 8 rows ahead in shared memory instead of one in registers, or two rows to an
// exchange, made it slower.
template <int DT, int WDT, int E, bool SECOND>
__global__ void __launch_bounds__(E == 24 ? 384 : kLnMaxThreads, E <= 24 ? 2 : 1)
    ln_forward_shifted(const __grid_constant__ LnForward a) {
  pdl_enter();
  constexpr uint32_t es = Elem<DT>::kSize, V = 16 / es, NV = E / V, H = V / 2;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) float slots[2][SECOND ? 3 : 2][kLnMaxThreads / 32];
  const uint32_t cols = (uint32_t)a.cols, t = threadIdx.x, group = blockDim.x;
  const char* base = static_cast<const char*>(a.x);
  const char* end = base + ((a.rows - 1) * a.x_stride + cols) * es;
  const uint32_t phase = line_phase(base + blockIdx.x * a.x_stride * es, es), lines = (phase + cols + V - 1) / V;
  // The CTA's rows have one phase, so what a thread's lines are is settled once: all inside the row, or on its edge.
  int at[NV];  // column of the line's first value
  uint32_t whole = 0, some = 0;
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
    at[j] = (int)((j * group + t) * V) - (int)phase;
    whole |= (at[j] >= 0 && at[j] + (int)V <= (int)cols ? 1u : 0u) << j;
    some |= (j * group + t < lines ? 1u : 0u) << j;
  }
  const char* x_next = base + blockIdx.x * a.x_stride * es;
  char* y = static_cast<char*>(a.y) + blockIdx.x * a.y_stride * es;
  const uint64_t x_hop = gridDim.x * a.x_stride * es, y_hop = gridDim.x * a.y_stride * es;
  uint4 q[NV];
  const auto fetch = [&]() {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      const char* line = x_next + at[j] * (int)es;
      if (whole >> j & 1u) q[j] = __ldcs(reinterpret_cast<const uint4*>(line));
      else if (some >> j & 1u) q[j] = load_line<DT>(line, base, end);
      else q[j] = make_uint4(0, 0, 0, 0);
    }
    x_next += x_hop;
  };
  fetch();
  float* ws = reinterpret_cast<float*>(smem);
  float* bs = ws + lines * V;
  for (uint32_t i0 = t; i0 < lines * V; i0 += 4 * group) {  // 8 reads in flight a thread
    float w[4], b[4];
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) {
      const uint32_t c = i0 + u * group - phase;  // wraps around before column 0
      w[u] = c >= cols ? 0.0f : a.w ? weight_at<WDT>(a.w, c) : 1.0f;
      b[u] = c < cols && a.b ? weight_at<WDT>(a.b, c) : 0.0f;
    }
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
      if (i0 + u * group < lines * V) {
        const uint32_t slot = weight_slot<V>(i0 + u * group, lines * 4);
        ws[slot] = w[u], bs[slot] = b[u];
      }
  }
  __syncthreads();
  const float n = (float)cols, inv_n = __frcp_rn(n);
  uint32_t parity = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, y += y_hop) {
    F2 f[E / 2], sum = 0;
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      widen<DT>(q[j], f + j * H);
      if (!(whole >> j & 1u)) mask_line<V>(f + j * H, -at[j], (int)cols - at[j]);
#pragma unroll
      for (uint32_t k = 0; k < H; ++k) sum = add2(sum, f[j * H + k]);
    }
    if (row + gridDim.x < a.rows) fetch();
    float mean = row_mean(cta_sum_registers(fold2(sum), slots[parity][0], group / 32), n, inv_n);
    if constexpr (SECOND) {
      const F2 minus = twice(-mean);
      F2 rest = 0;
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        F2 d[H];
#pragma unroll
        for (uint32_t k = 0; k < H; ++k) d[k] = add2(f[j * H + k], minus);
        if (!(whole >> j & 1u)) mask_line<V>(d, -at[j], (int)cols - at[j]);
#pragma unroll
        for (uint32_t k = 0; k < H; ++k) rest = add2(rest, d[k]);
      }
      mean += mean_rest(row_mean(cta_sum_registers(fold2(rest), slots[parity][2], group / 32), n, inv_n));
    }
    const F2 minus = twice(-mean);
    F2 sq = 0;
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
#pragma unroll
      for (uint32_t k = 0; k < H; ++k) f[j * H + k] = add2(f[j * H + k], minus);
      if (!(whole >> j & 1u)) mask_line<V>(f + j * H, -at[j], (int)cols - at[j]);
#pragma unroll
      for (uint32_t k = 0; k < H; ++k) sq = fma2(f[j * H + k], f[j * H + k], sq);
    }
    const float var = cta_sum_registers(fold2(sq), slots[parity][1], group / 32) * inv_n;
    const float rstd = rsqrtf(var + a.eps);
    const F2 rstd2 = twice(rstd);
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      if (!(some >> j & 1u)) continue;
      const uint32_t first = (j * group + t) * 4;
#pragma unroll
      for (uint32_t e = 0; e < H; e += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(ws + first + e / 2 * lines * 4);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(bs + first + e / 2 * lines * 4);
        f[j * H + e] = fma2(mul2(f[j * H + e], rstd2), w.x, b.x);
        f[j * H + e + 1] = fma2(mul2(f[j * H + e + 1], rstd2), w.y, b.y);
      }
      const uint4 out = narrow<DT>(f + j * H);
      if (whole >> j & 1u) __stcs(reinterpret_cast<uint4*>(y + at[j] * (int)es), out);
      else store_part<DT>(y + at[j] * (int)es, out, -at[j], (int)cols - at[j]);
    }
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    parity ^= 1;
  }
}

// ---- the backward pass in one sweep --------------------------------------------
// One CTA per SM; its groups of threads walk over the rows. The next rows of x
// and dy are on their way into shared memory (cp.async, up to 8 rows ahead)
// while one is worked on, and the column sums of dy xhat and dy stay in
// registers over all the rows of a group: x and dy are read once. The CTA folds
// its groups' sums and writes one partial of each; ln_backward_finish adds the
// partials (a CTA that has all the rows writes the gradients itself). KEEP: xhat
// and dy w of the row stay in registers between their two uses (before and after
// the row's sums), and its place in shared memory is filled again at once;
// otherwise they are taken from shared memory twice.
//
// SHIFTED: rows off the 16-byte grid, by whole lines as above. The rows of a
// CTA are a multiple of 8 apart, so all of them have the same phase and a
// register keeps standing for the same column.
//
// LATE: a row too long for one CTA's registers or shared memory is shared by the
// 2 or 4 CTAs of a cluster, each with a run of its lines; their sums meet in
// each other's shared memory, and a row's dx waits until the next row's sums are
// on their way. 4096 x 20000 bf16: 132 us (55% of the copy bandwidth), 4096 x
// 16384 fp32: 141 us (84%), against 500 and 459 us in separate passes for dx and
// the column sums; without the delay 233 and 171.
//
// Measured (back to back, inputs larger than L2, of the copy bandwidth's floor):
// 8192 x 1024 bf16 15.7 us (7.4), of which about 3 are the first rows' way, 9 the
// loop at 80% of the copy bandwidth, 1 the fold and 2 ln_backward_finish; 32768 x
// 8192 bf16 286 us (237); 2047 x 1537 fp32 14.3 us (5.6); 6001 x 4095 fp16 59 us
// (21.7). In the loop 16 warps (accumulators and the row's values fill the
// registers) keep 40 to 45% of the issue slots busy: the chain from the row's
// sums through the exchange to dx bounds it as much as HBM does.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  // copies `bytes` (0 to 16) and fills up with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Waits until all but the stages - 1 newest groups of copies have landed, or fewer; stages: 1 to 8.
__device__ __forceinline__ void cp_async_wait_oldest(uint32_t stages) {
  if (stages == 8) cp_async_wait<7>();
  else if (stages >= 6) cp_async_wait<5>();
  else if (stages >= 4) cp_async_wait<3>();
  else if (stages == 3) cp_async_wait<2>();
  else if (stages == 2) cp_async_wait<1>();
  else cp_async_wait<0>();
}

// The CTAs of a cluster: all of their threads, and a float to another CTA's shared memory at the address that `at`
// has in this one's.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_in_cluster(const float* at, uint32_t rank, float v) {
  const uint32_t local = (uint32_t)__cvta_generic_to_shared(at);
  asm volatile(
      "{\n .reg .b32 there;\n mapa.shared::cluster.u32 there, %0, %1;\n st.shared::cluster.f32 [there], %2;\n}" ::"r"(local),
      "r"(rank), "f"(v)
      : "memory");
}

// All threads of a row's group: a named barrier of its own, or the warp.
__device__ __forceinline__ void group_sync(uint32_t g, uint32_t size) {
  if (size == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(size) : "memory");
}

// Elements of one row's lines, and of a CTA's share of them, in shared memory.
__host__ __device__ constexpr uint32_t ln_share_elems(uint32_t cols, uint32_t es, bool shifted, uint32_t ranks) {
  return ((cols + (shifted ? 16 / es - 1 : 0) + 16 / es - 1) / (16 / es) + ranks - 1) / ranks * (16 / es);
}

// Column c's sums to where they go.
template <int WDT>
__device__ __forceinline__ void finish_column(const LnBackward& a, uint64_t c, float dw, float db) {
  if (a.dw) ln_store<WDT>(a.dw, c, a.accumulate ? ln_load<WDT>(a.dw, c) + dw : dw);
  if (a.db) ln_store<WDT>(a.db, c, a.accumulate ? ln_load<WDT>(a.db, c) + db : db);
}

template <int DT, int WDT, int E, bool KEEP, bool SHIFTED, bool LATE>
__global__ void __launch_bounds__(kLnMaxThreads, 1) ln_backward_fused(const __grid_constant__ LnBackward a) {
  pdl_enter();
  constexpr uint32_t es = Elem<DT>::kSize, V = 16 / es, NV = E / V, H = V / 2;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) float2 slots[2][(LATE ? kLnMaxSplit : 1) * kLnMaxThreads / 32];
  const uint32_t cols = (uint32_t)a.cols, size = a.group, groups = blockDim.x / size, stages = a.stages;
  const uint32_t g = threadIdx.x / size, t = threadIdx.x - g * size, lane = threadIdx.x & 31;
  uint32_t rank = 0, ranks = 1, unit = blockIdx.x, units = gridDim.x;
  if constexpr (LATE) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    ranks = a.split, unit = blockIdx.x / ranks, units = gridDim.x / ranks;
  }
  const uint32_t row_elems = ln_share_elems(cols, es, SHIFTED, ranks), row_bytes = row_elems * es;
  const uint32_t half = row_elems / 2;  // from a line's first four weights to its second four
  float* weights = reinterpret_cast<float*>(smem);
  char* ring = smem + row_elems * 4 + (size_t)g * stages * 2 * row_bytes;

  // few rows spread over the CTAs first, then over their groups
  const uint64_t first = (uint64_t)g * units + unit, stride = (uint64_t)units * groups;
  const char* xs = static_cast<const char*>(a.x);
  const char* dys = static_cast<const char*>(a.dy);
  const uint32_t phase = SHIFTED ? line_phase(xs + unit * a.x_stride * es, es) : 0;
  const uint32_t all_lines = (phase + cols + V - 1) / V, line0 = rank * (row_elems / V);  // of the row, and of this CTA's share
  const uint32_t lines = LATE ? (all_lines > line0 ? min(all_lines - line0, row_elems / V) : 0) : all_lines;
  const int column0 = (int)(line0 * V) - (int)phase;  // of the share's first line
  const char* x_end = xs + ((a.rows - 1) * a.x_stride + cols) * es;
  const char* dy_end = dys + ((a.rows - 1) * a.dy_stride + cols) * es;
  // this thread's first lines of the next row to fetch, the row itself, and where they go
  const char* x_next = xs + first * a.x_stride * es - phase * es + (line0 + t) * 16;
  const char* dy_next = dys + first * a.dy_stride * es - phase * es + (line0 + t) * 16;
  const uint64_t x_hop = stride * a.x_stride * es, dy_hop = stride * a.dy_stride * es, dx_hop = stride * a.dx_stride * es;
  uint64_t row_next = first;
  const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  const auto fetch_lines = [&](uint32_t dst, const char* line, const char* base, const char* end) {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      if (j * size + t >= lines) continue;
      const char* at = line + j * size * 16;
      const uint32_t to = dst + j * size * 16;
      if constexpr (!SHIFTED) {
        cp_async16(to, at, 16);
      } else if (at >= base) {
        const uint64_t left = (uint64_t)(end - at);
        cp_async16(to, at, left < 16 ? (uint32_t)left : 16);
      } else {  // the matrix starts inside this line
        const uint4 q = load_line<DT>(at, base, end);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
      }
    }
  };
  const auto fetch = [&](uint32_t stage) {
    if (row_next < a.rows) {
      const uint32_t dst = mine_at + stage * 2 * row_bytes;
      fetch_lines(dst, x_next, xs, x_end);
      fetch_lines(dst + row_bytes, dy_next, dys, dy_end);
      x_next += x_hop, dy_next += dy_hop, row_next += stride;
    }
    cp_async_commit();
  };
  // The weights and the first row's statistics are asked for before the rows: behind 200 KB of them per SM they
  // would arrive last, and nothing could begin (6 us of 17 at 8192 x 1024 bf16).
  float mean = 0.0f, rstd = 0.0f;
  if (first < a.rows) mean = __ldg(a.mean + first), rstd = __ldg(a.rstd + first);
  // one row ahead, or two where registers allow (4096 x 12288 bf16: 101 -> 78 us; at E = 16 it costs 1%)
  constexpr uint32_t kAhead = E == 16 ? 1 : 2;
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (kAhead == 2 && first + stride < a.rows)
    next_mean = __ldg(a.mean + first + stride), next_rstd = __ldg(a.rstd + first + stride);
  const auto weight = [&](uint32_t i) {
    const uint32_t c = (uint32_t)(column0 + (int)i);  // wraps around before column 0
    return c >= cols ? 0.0f : a.w ? weight_at<WDT>(a.w, c) : 1.0f;
  };
  constexpr uint32_t kEarly = 4;
  for (uint32_t i0 = threadIdx.x + kEarly * blockDim.x; i0 < row_elems; i0 += 8 * blockDim.x) {  // 8 reads in flight
    float w[8];
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u) w[u] = i0 + u * blockDim.x < row_elems ? weight(i0 + u * blockDim.x) : 0.0f;
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u)
      if (i0 + u * blockDim.x < row_elems) weights[weight_slot<V>(i0 + u * blockDim.x, half)] = w[u];
  }
  float early[kEarly];
#pragma unroll
  for (uint32_t k = 0; k < kEarly; ++k) {
    const uint32_t i = threadIdx.x + k * blockDim.x;
    early[k] = i < row_elems ? weight(i) : 0.0f;
  }
  for (uint32_t s = 0; s < stages; ++s) fetch(s);
#pragma unroll
  for (uint32_t k = 0; k < kEarly; ++k) {
    const uint32_t i = threadIdx.x + k * blockDim.x;
    if (i < row_elems) weights[weight_slot<V>(i, half)] = early[k];
  }
  if constexpr (LATE) cluster_sync();  // the others' shared memory is there
  else __syncthreads();

  F2 dw[E / 2], db[E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) dw[k] = db[k] = 0;
  const float inv_n = 1.0f / (float)cols;
  uint32_t stage = 0, parity = 0;
  const char* buffer = ring + t * 16;  // this thread's first line of the row in work
  const float* w_at = weights + t * 4;
  char* dx = static_cast<char*>(a.dx) + first * a.dx_stride * es - phase * es + (line0 + t) * 16;
  // xhat, dy and the weights of the thread's j-th line of the row in `buffer`. The mean is subtracted before anything
  // is rounded (x rstd - mean rstd in one fused operation would be off by mean rstd's own rounding: 1e-3 of xhat where
  // the mean is 10,000 deviations).
  const auto load = [&](const char* buffer, F2 rstd2, F2 minus_mean2, uint32_t j, F2* h, F2* dy, F2* w) {
    widen<DT>(*reinterpret_cast<const uint4*>(buffer + j * size * 16), h);
    widen<DT>(*reinterpret_cast<const uint4*>(buffer + row_bytes + j * size * 16), dy);
#pragma unroll
    for (uint32_t e = 0; e < H; ++e) h[e] = mul2(add2(h[e], minus_mean2), rstd2);
    if constexpr (SHIFTED) {
      const int at = column0 + (int)((j * size + t) * V);
      if (at < 0 || at + (int)V > (int)cols) mask_line<V>(h, -at, (int)cols - at), mask_line<V>(dy, -at, (int)cols - at);
    }
#pragma unroll
    for (uint32_t e = 0; e < H; e += 2) {
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(w_at + j * size * 4 + e / 2 * half);
      w[e] = q.x, w[e + 1] = q.y;
    }
  };
  const auto store = [&](char* dx, uint32_t j, const F2* out) {
    const uint4 q = narrow<DT>(out);
    const int at = column0 + (int)((j * size + t) * V);
    if (!SHIFTED || (at >= 0 && at + (int)V <= (int)cols)) __stcs(reinterpret_cast<uint4*>(dx + j * size * 16), q);
    else store_part<DT>(dx + j * size * 16, q, -at, (int)cols - at);
  };
  if constexpr (LATE) {
    // A row's dx waits until the next row's sums are on their way, so that the exchange between the warps (and CTAs)
    // is hidden behind it; its place in shared memory is filled again after that.
    const char* old_buffer = nullptr;
    char* old_dx = nullptr;
    uint32_t old_stage = 0;
    F2 old_rstd2 = 0, old_minus_mean2 = 0, old_c1 = 0, old_c2 = 0;
    const auto late_dx = [&]() {
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        if (j * size + t >= lines) continue;
        F2 out[H], dy[H], w[H];
        load(old_buffer, old_rstd2, old_minus_mean2, j, out, dy, w);
#pragma unroll
        for (uint32_t e = 0; e < H; ++e) out[e] = fma2(mul2(dy[e], w[e]), old_rstd2, fma2(out[e], old_c2, old_c1));
        store(old_dx, j, out);
      }
      fetch(old_stage);
    };
    const uint32_t warps = size / 32;
    for (uint64_t row = first; row < a.rows; row += stride, dx += dx_hop) {
      cp_async_wait_oldest(stages - 1);  // the place of the row before is not sent for yet
      float new_mean = 0.0f, new_rstd = 0.0f;
      if (row + kAhead * stride < a.rows)
        new_mean = __ldg(a.mean + row + kAhead * stride), new_rstd = __ldg(a.rstd + row + kAhead * stride);
      const F2 rstd2 = twice(rstd), minus_mean2 = twice(-mean);
      F2 sum1 = 0, sum2 = 0;
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        if (j * size + t >= lines) continue;
        F2 h[H], dy[H], w[H];
        load(buffer, rstd2, minus_mean2, j, h, dy, w);
#pragma unroll
        for (uint32_t e = 0; e < H; ++e) {
          const F2 p = mul2(dy[e], w[e]);
          sum1 = add2(sum1, p);
          sum2 = fma2(p, h[e], sum2);
          dw[j * H + e] = fma2(dy[e], h[e], dw[j * H + e]);
          db[j * H + e] = add2(db[j * H + e], dy[e]);
        }
      }
      float s1 = fold2(sum1), s2 = fold2(sum2);
      const bool up = lane & 16;  // the lower half of a warp carries one sum, the upper the other
      float mine = (up ? s2 : s1) + __shfl_xor_sync(0xffffffffu, up ? s1 : s2, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      if ((lane & 15) < ranks)
        store_in_cluster(reinterpret_cast<const float*>(&slots[parity][rank * warps + threadIdx.x / 32]) + lane / 16,
                         lane & 15, mine);
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      if (old_buffer != nullptr) late_dx();
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      s1 = s2 = 0.0f;
      for (uint32_t k = lane; k < ranks * warps; k += 32) s1 += slots[parity][k].x, s2 += slots[parity][k].y;
      s1 = warp_sum(s1), s2 = warp_sum(s2);
      parity ^= 1;
      old_rstd2 = rstd2, old_minus_mean2 = minus_mean2, old_c1 = twice(-rstd * (s1 * inv_n)), old_c2 = twice(-rstd * (s2 * inv_n));
      old_buffer = buffer, old_dx = dx, old_stage = stage;
      if constexpr (kAhead == 1) mean = new_mean, rstd = new_rstd;
      else mean = next_mean, rstd = next_rstd, next_mean = new_mean, next_rstd = new_rstd;
      ++stage, buffer += 2 * row_bytes;
      if (stage == stages) stage = 0, buffer = ring + t * 16;
    }
    if (old_buffer != nullptr) late_dx();
  } else {
    for (uint64_t row = first; row < a.rows; row += stride, dx += dx_hop) {
      cp_async_wait_oldest(stages);  // every thread reads back the lines it fetched itself: nothing else to wait for
      float new_mean = 0.0f, new_rstd = 0.0f;
      if (row + kAhead * stride < a.rows)
        new_mean = __ldg(a.mean + row + kAhead * stride), new_rstd = __ldg(a.rstd + row + kAhead * stride);
      const F2 rstd2 = twice(rstd), minus_mean2 = twice(-mean);
      F2 hs[KEEP ? E / 2 : 1], ps[KEEP ? E / 2 : 1], sum1 = 0, sum2 = 0;
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        if (j * size + t >= lines) continue;
        F2 h[H], dy[H], w[H];
        load(buffer, rstd2, minus_mean2, j, h, dy, w);
#pragma unroll
        for (uint32_t e = 0; e < H; ++e) {
          const F2 p = mul2(dy[e], w[e]);
          sum1 = add2(sum1, p);
          sum2 = fma2(p, h[e], sum2);
          dw[j * H + e] = fma2(dy[e], h[e], dw[j * H + e]);
          db[j * H + e] = add2(db[j * H + e], dy[e]);
          if constexpr (KEEP) hs[j * H + e] = h[e], ps[j * H + e] = p;
        }
      }
      if constexpr (KEEP) fetch(stage);
      // both sums in one exchange: the lower half of a warp carries one, the upper the other
      float s1 = fold2(sum1), s2 = fold2(sum2);
      {
        const bool up = lane & 16;
        float mine = (up ? s2 : s1) + __shfl_xor_sync(0xffffffffu, up ? s1 : s2, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (size > 32) {
          const uint32_t warps = size / 32;
          if ((lane & 15) == 0) reinterpret_cast<float*>(&slots[parity][threadIdx.x / 32])[lane / 16] = mine;
          group_sync(g, size);
          if (warps <= 8) {  // all read them: no second round of shuffles (which is faster for 16 warps)
            const F2* all = reinterpret_cast<const F2*>(&slots[parity][g * warps]);
            F2 even = 0, odd = 0;
#pragma unroll
            for (uint32_t k = 0; k < 8; k += 2) {
              if (k >= warps) break;
              even = add2(even, all[k]);
              if (k + 1 < warps) odd = add2(odd, all[k + 1]);
            }
            split(add2(even, odd), s1, s2);
          } else {
            const uint32_t w = lane & 15;
            mine = w < warps ? reinterpret_cast<const float*>(&slots[parity][g * warps + w])[lane / 16] : 0.0f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
            s1 = __shfl_sync(0xffffffffu, mine, 0), s2 = __shfl_sync(0xffffffffu, mine, 16);
          }
          parity ^= 1;
        } else {
          s1 = __shfl_sync(0xffffffffu, mine, 0), s2 = __shfl_sync(0xffffffffu, mine, 16);
        }
      }
      // rstd (p - s1/n - xhat s2/n)
      const float c1 = -rstd * (s1 * inv_n), c2 = -rstd * (s2 * inv_n);
      const F2 c1_2 = pair(c1, c1), c2_2 = pair(c2, c2);
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        if (j * size + t >= lines) continue;
        F2 out[H];
        if constexpr (KEEP) {
#pragma unroll
          for (uint32_t e = 0; e < H; ++e) out[e] = fma2(ps[j * H + e], rstd2, fma2(hs[j * H + e], c2_2, c1_2));
        } else {
          F2 dy[H], w[H];
          load(buffer, rstd2, minus_mean2, j, out, dy, w);
#pragma unroll
          for (uint32_t e = 0; e < H; ++e) out[e] = fma2(mul2(dy[e], w[e]), rstd2, fma2(out[e], c2_2, c1_2));
        }
        store(dx, j, out);
      }
      if constexpr (!KEEP) fetch(stage);
      if constexpr (kAhead == 1) mean = new_mean, rstd = new_rstd;
      else mean = next_mean, rstd = next_rstd, next_mean = new_mean, next_rstd = new_rstd;
      ++stage, buffer += 2 * row_bytes;
      if (stage == stages) stage = 0, buffer = ring + t * 16;
    }
  }
  if constexpr (LATE) cluster_sync();  // no CTA leaves while another may still write to it
  if (a.dw == nullptr && a.db == nullptr) return;
  // fold the groups: every group's sums side by side in shared memory, then column by column
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
    const uint32_t k = j * size + t;
    if (k >= lines) continue;
    float* to = sums + g * 2 * row_elems + k * V;
#pragma unroll
    for (uint32_t e = 0; e < H; e += 2) {
      *reinterpret_cast<ulonglong2*>(to + 2 * e) = make_ulonglong2(dw[j * H + e], dw[j * H + e + 1]);
      *reinterpret_cast<ulonglong2*>(to + row_elems + 2 * e) = make_ulonglong2(db[j * H + e], db[j * H + e + 1]);
    }
  }
  __syncthreads();
  float* part = a.part + (uint64_t)unit * 2 * cols;
  const uint32_t from = column0 < 0 ? (uint32_t)-column0 : 0;  // of the share, not before column 0
  for (uint32_t i = from + threadIdx.x; i < lines * V && column0 + (int)i < (int)cols; i += blockDim.x) {
    float w = 0.0f, b = 0.0f;
    for (uint32_t k = 0; k < groups; ++k) {
      w += sums[k * 2 * row_elems + i];
      b += sums[(k * 2 + 1) * row_elems + i];
    }
    const uint64_t c = (uint64_t)(column0 + (int)i);
    if (a.parts > 1) part[c] = w, part[cols + c] = b;
    else finish_column<WDT>(a, c, w, b);
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
  const bool second = second_mean<DT>(a.cols);
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + row * a.x_stride * es;
    char* y = static_cast<char*>(a.y) + row * a.y_stride * es;
    float sum = 0.0f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) sum += ln_load<DT>(x, i);
    float mean = __fdiv_rn(cta_sum_all<kLnThreads>(sum, smem), n);
    if (second) {
      float rest = 0.0f;
      for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) rest += ln_load<DT>(x, i) - mean;
      mean += mean_rest(__fdiv_rn(cta_sum_all<kLnThreads>(rest, smem), n));
    }
    float sq = 0.0f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kLnThreads) {
      const float d = ln_load<DT>(x, i) - mean;
      sq = __fmaf_rn(d, d, sq);
    }
    const float var = __fdiv_rn(cta_sum_all<kLnThreads>(sq, smem), n);
    const float rstd = rsqrtf(var + a.eps);
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

// The sums of the partials: CTA x takes 32 columns, each warp a share of the parts. All of a thread's reads are
// independent and there are few of them: the kernel is one trip to L2 and back.
constexpr int kLnFinishThreads = 1024;
template <int WDT>
__global__ void __launch_bounds__(kLnFinishThreads) ln_backward_finish(const __grid_constant__ LnBackward a) {
  pdl_enter();
  constexpr int kWarps = kLnFinishThreads / 32, kReads = ((int)kLnMaxParts + kWarps - 1) / kWarps;
  __shared__ float sw[kWarps][33], sb[kWarps][33];
  const int lane = threadIdx.x & 31, wid = threadIdx.x / 32;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  float w[kReads], b[kReads];
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    const int p = k * kWarps + wid;
    const bool in = p < a.parts && c < a.cols;
    w[k] = in ? __ldcg(a.part + (uint64_t)p * 2 * a.cols + c) : 0.0f;
    b[k] = in ? __ldcg(a.part + ((uint64_t)p * 2 + 1) * a.cols + c) : 0.0f;
  }
#pragma unroll
  for (int k = 1; k < kReads; ++k) w[0] += w[k], b[0] += b[k];
  sw[wid][lane] = w[0], sb[wid][lane] = b[0];
  __syncthreads();
  // warp q sums column q of the block's 32: over the warps, in the same tree every time
  float dw = sw[lane][wid], db = sb[lane][wid];
  dw = warp_sum(dw), db = warp_sum(db);
  const uint64_t mine = (uint64_t)blockIdx.x * 32 + wid;
  if (lane == 0 && mine < a.cols) finish_column<WDT>(a, mine, dw, db);
}

}  // namespace ra
