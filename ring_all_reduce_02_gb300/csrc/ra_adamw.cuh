// AdamW over many tensors in one launch, moments in fp32 or in 8 bits.
//
// Per element (g the scaled gradient, all fp32, every product and sum rounded):
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// It touches every byte once, so HBM bounds it: 4 + 4 + 2 + 8 + 8 + 2 = 28
// bytes per element for fp32 parameters and moments with bf16 gradients and
// copies, 10 for bf16 parameters with 8-bit moments.
//
// Work: a warp takes chunks of 256 consecutive elements, 8 per lane. With 8-bit
// moments a chunk is one block of the scales, so the block's largest magnitude
// is one warp reduction and the moments never leave registers between being
// read and being stored again. The tensors' table travels in the kernel's
// parameters; a CTA finds its tensor by bisection over the tensors' first CTAs.
#pragma once

#include <cuda_fp8.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"

namespace ra {

constexpr int kAdamBlock = 256;  // elements per chunk, and per scale of an 8-bit moment
constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  void* copy;
  uint64_t count;
  float keep;       // 1 - lr * weight_decay
  uint32_t layout;  // kAdamVec: every buffer has vectors of 8 elements at elements 8 k - shift; low 3 bits: shift
};
constexpr uint32_t kAdamVec = 8;

// Kernel parameters hold at most 32,764 bytes; the small table keeps short lists' launches short.
constexpr int kAdamSmall = 16;
constexpr int kAdamLarge = 416;

struct AdamScalars {
  float b1, one_minus_b1, b2, one_minus_b2, inv_sqrt_bc2, eps, step_size;
  int n;              // tensors in the table
  uint32_t key;       // of the random bits
  uint32_t ordinal0;  // place of table entry 0 in the caller's list
  int copy_dtype;
  const float* scale;
};
template <int CAP>
struct AdamArgs {
  AdamScalars s;
  uint32_t cta0[CAP];  // first CTA of each tensor
  AdamTensor t[CAP];
};

// A 32-bit mix: xor-shifts and multiplications by odd constants (the fractions of e and of the golden ratio).
__host__ __device__ __forceinline__ uint32_t mix32_but_last(uint32_t x) {
  x ^= x >> 16;
  x *= 0xB7E15163u;
  x ^= x >> 15;
  return x * 0x9E3779B9u;
}
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = mix32_but_last(x);
  return x ^ (x >> 16);
}
// The 16 low and the 16 high bits of mix32, each 4 places up, from mix32_but_last.
__device__ __forceinline__ uint32_t low_bits(uint32_t x) { return ((x << 4) ^ (x >> 12)) & 0xffff0u; }
__device__ __forceinline__ uint32_t high_bits(uint32_t x) { return (x >> 12) & 0xffff0u; }

template <int DT>
__device__ __forceinline__ float load_as_f32(const void* base, uint64_t i) {
  if constexpr (DT == DT_F32) return __ldcs(static_cast<const float*>(base) + i);
  else return widen16<DT>(ld_elem<DT>(base, i));
}
template <int DT>
__device__ __forceinline__ void store_f32_as(void* base, uint64_t i, float x) {
  if constexpr (DT == DT_F32) __stcs(static_cast<float*>(base) + i, x);
  else st_elem<DT>(base, i, round16<DT>(x));
}
__device__ __forceinline__ float load_e4m3(const void* base, uint64_t i) {
  const __nv_fp8_storage_t b = __ldcs(static_cast<const unsigned char*>(base) + i);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// A value scaled to its block (x * 448 / amax), rounded up or down in e4m3's normal range by 16 random bits in
// places 4 to 19: the bits below the 3 kept ones of the mantissa decide with their own weight. The conversion
// that follows saturates, so that nothing passes 448.
__device__ __forceinline__ float round_up_or_down(float x, uint32_t bits) {
  return __uint_as_float((__float_as_uint(x) + bits) & 0xfff00000u);
}

// 8 consecutive elements at element i, as fp32; i and the base are on the 8-element grid.
template <int DT>
__device__ __forceinline__ void load8(const void* base, uint64_t i, float* f) {
  if constexpr (DT == DT_F32) {
    const VecT<8> v = ld_vec_w<8>(static_cast<const float*>(base) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v.w[k]);
  } else {
    const VecT<4> v = ld_vec_w<4>(static_cast<const unsigned short*>(base) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = widen16<DT>((v.w[k / 2] >> (k % 2 * 16)) & 0xffffu);
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* base, uint64_t i, const float* f) {
  if constexpr (DT == DT_F32) {
    VecT<8> v;
#pragma unroll
    for (int k = 0; k < 8; ++k) v.w[k] = __float_as_uint(f[k]);
    st_vec<8>(static_cast<float*>(base) + i, v);
  } else {
    VecT<4> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v.w[k] = round16<DT>(f[2 * k]) | round16<DT>(f[2 * k + 1]) << 16;
    st_vec<4>(static_cast<unsigned short*>(base) + i, v);
  }
}
__device__ __forceinline__ void load8_e4m3(const void* base, uint64_t i, float* f) {
  const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(base) + i));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((k < 2 ? q.x : q.y) >> (k % 2 * 16));
    const float2 p = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    f[2 * k] = p.x, f[2 * k + 1] = p.y;
  }
}
__device__ __forceinline__ uint32_t pack4_e4m3(const float* f) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ void sum_rn(F2 x, F2 y, float& a, float& b) {
  float x0, x1, y0, y1;
  split(x, x0, x1), split(y, y0, y1);
  a = __fadd_rn(x0, y0), b = __fadd_rn(x1, y1);
}

// One chunk of a tensor by one warp: elements base .. base + 255, of which [0, count) exist. WHOLE: all of them
// do, on the 8-element grid of every buffer, and lane l takes 8 l .. 8 l + 7; otherwise lane l takes l, l + 32, ...
template <int P, int G, bool S8, bool WHOLE>
__device__ __forceinline__ void adamw_chunk(const AdamScalars& s, const AdamTensor& t, int64_t base, uint64_t chunk,
                                            uint32_t key, float scale) {
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t i0 = (uint64_t)base + (WHOLE ? 8 * lane : 0);
  const auto at = [&](int j) { return base + (int64_t)lane + 32 * j; };
  const auto in = [&](int j) { return (uint64_t)at(j) < t.count; };  // a negative place wraps around
  float p[8], g[8], m[8], r[8];  // r: v, then its square root
  float m_scale = 0.0f, r_scale = 0.0f;
  if constexpr (S8) m_scale = t.ms[chunk], r_scale = t.vs[chunk];
  if constexpr (WHOLE) {
    load8<G>(t.g, i0, g);
    load8<P>(t.p, i0, p);
    if constexpr (S8) load8_e4m3(t.m, i0, m), load8_e4m3(t.v, i0, r);
    else load8<DT_F32>(t.m, i0, m), load8<DT_F32>(t.v, i0, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = in(j) ? load_as_f32<G>(t.g, at(j)) : 0.0f;
      p[j] = in(j) ? load_as_f32<P>(t.p, at(j)) : 0.0f;
      if constexpr (S8) m[j] = in(j) ? load_e4m3(t.m, at(j)) : 0.0f, r[j] = in(j) ? load_e4m3(t.v, at(j)) : 0.0f;
      else m[j] = in(j) ? load_as_f32<DT_F32>(t.m, at(j)) : 0.0f, r[j] = in(j) ? load_as_f32<DT_F32>(t.v, at(j)) : 0.0f;
    }
  }
  const F2 scale2 = twice(scale), b1 = twice(s.b1), b1c = twice(s.one_minus_b1), b2 = twice(s.b2), b2c = twice(s.one_minus_b2);
  const F2 bc = twice(s.inv_sqrt_bc2), eps = twice(s.eps), keep = twice(t.keep), step = twice(-s.step_size);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const F2 gg = mul2(pair(g[j], g[j + 1]), scale2);
    F2 mm = pair(m[j], m[j + 1]), vv = pair(r[j], r[j + 1]);
    if constexpr (S8) mm = mul2(mm, twice(m_scale)), vv = mul2(vv, twice(r_scale)), vv = mul2(vv, vv);
    // products and sums rounded one by one: the stored moments are the same bits as the formula's written out
    // (the sums are scalar: the assembler contracts a mul.f32x2 and an add.f32x2, rounding modifiers or not)
    sum_rn(mul2(mm, b1), mul2(gg, b1c), m[j], m[j + 1]);
    sum_rn(mul2(vv, b2), mul2(mul2(gg, b2c), gg), r[j], r[j + 1]);
    const float r0 = __fsqrt_rn(r[j]), r1 = __fsqrt_rn(r[j + 1]);
    float d0, d1;
    split(fma2(pair(r0, r1), bc, eps), d0, d1);
    const F2 u = pair(__fdividef(m[j], d0), __fdividef(m[j + 1], d1));
    split(fma2(u, step, mul2(pair(p[j], p[j + 1]), keep)), p[j], p[j + 1]);
    if constexpr (S8) r[j] = r0, r[j + 1] = r1;
  }
  if constexpr (WHOLE) {
    store8<P>(t.p, i0, p);
    if constexpr (!S8) store8<DT_F32>(t.m, i0, m), store8<DT_F32>(t.v, i0, r);
    if (t.copy != nullptr) {
      if (s.copy_dtype == DT_F32) store8<DT_F32>(t.copy, i0, p);
      else if (s.copy_dtype == DT_F16) store8<DT_F16>(t.copy, i0, p);
      else store8<DT_BF16>(t.copy, i0, p);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!in(j)) continue;
      store_f32_as<P>(t.p, at(j), p[j]);
      if constexpr (!S8) store_f32_as<DT_F32>(t.m, at(j), m[j]), store_f32_as<DT_F32>(t.v, at(j), r[j]);
      if (t.copy != nullptr) {
        if (s.copy_dtype == DT_F32) store_f32_as<DT_F32>(t.copy, at(j), p[j]);
        else if (s.copy_dtype == DT_F16) store_f32_as<DT_F16>(t.copy, at(j), p[j]);
        else store_f32_as<DT_BF16>(t.copy, at(j), p[j]);
      }
    }
  }
  if constexpr (S8) {
    float m_top = 0.0f, r_top = 0.0f;  // NaN wins, and its bits are above infinity's
#pragma unroll
    for (int j = 0; j < 8; ++j) m_top = fmaximum(m_top, fabsf(m[j])), r_top = fmaximum(r_top, r[j]);
    const float m_amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m_top)));
    const float r_amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r_top)));
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);
    const bool m_some = m_amax > kMinAmax, r_some = r_amax > kMinAmax;
    const bool m_bad = !(m_amax < inf), r_bad = !(r_amax < inf);
    const float m_inv = m_some ? __frcp_rn(m_amax) * kE4m3Max : 0.0f;
    const float r_inv = r_some ? __frcp_rn(r_amax) * kE4m3Max : 0.0f;
    if (lane == 0) {
      t.ms[chunk] = m_bad ? nan : m_some ? m_amax * (1.0f / kE4m3Max) : 0.0f;
      t.vs[chunk] = r_bad ? nan : r_some ? r_amax * (1.0f / kE4m3Max) : 0.0f;
    }
    const float r_floor = r_some ? 0.001953125f : 0.0f;  // 2^-9, the smallest value above zero
    const uint32_t seed0 = (uint32_t)i0 * 0x9E3779B9u + (uint32_t)(i0 >> 32) * 0xB7E15163u + key;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t rand[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint64_t i = (uint64_t)at(j + k);
        rand[k] = mix32_but_last(WHOLE ? seed0 + (j + k) * 0x9E3779B9u  // 8 elements from a multiple of 8 share i >> 32
                                       : (uint32_t)i * 0x9E3779B9u + (uint32_t)(i >> 32) * 0xB7E15163u + key);
      }
      split(mul2(pair(m[j], m[j + 1]), twice(m_inv)), m[j], m[j + 1]);
      float t0, t1;
      split(mul2(pair(r[j], r[j + 1]), twice(r_inv)), t0, t1);
      m[j] = round_up_or_down(m[j], low_bits(rand[0])), m[j + 1] = round_up_or_down(m[j + 1], low_bits(rand[1]));
      t0 = round_up_or_down(t0, high_bits(rand[0])), t1 = round_up_or_down(t1, high_bits(rand[1]));
      if (r[j] > 0.0f) t0 = fmaxf(t0, r_floor);
      if (r[j + 1] > 0.0f) t1 = fmaxf(t1, r_floor);
      r[j] = t0, r[j + 1] = t1;
    }
    if constexpr (WHOLE) {
      uint2 mq = make_uint2(pack4_e4m3(m), pack4_e4m3(m + 4)), rq = make_uint2(pack4_e4m3(r), pack4_e4m3(r + 4));
      if (m_bad) mq = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      if (r_bad) rq = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      __stcs(reinterpret_cast<uint2*>(static_cast<unsigned char*>(t.m) + i0), mq);
      __stcs(reinterpret_cast<uint2*>(static_cast<unsigned char*>(t.v) + i0), rq);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!in(j)) continue;
        static_cast<unsigned char*>(t.m)[at(j)] = m_bad ? 0x7f : __nv_cvt_float_to_fp8(m[j], __NV_SATFINITE, __NV_E4M3);
        static_cast<unsigned char*>(t.v)[at(j)] = r_bad ? 0x7f : __nv_cvt_float_to_fp8(r[j], __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

template <int P, int G, bool S8, int CAP>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamArgs<CAP> a) {
  pdl_enter();
  const AdamScalars& s = a.s;
  float scale = 1.0f;
  if (s.scale != nullptr) {
    scale = *s.scale;
    if (!(fabsf(scale) < __int_as_float(0x7f800000))) return;  // not finite: the step is skipped
  }
  int lo = 0, hi = s.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cta0[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamTensor& t = a.t[lo];
  const uint64_t chunk = (uint64_t)(blockIdx.x - a.cta0[lo]) * kAdamWarps + threadIdx.x / 32;
  const int64_t base = (int64_t)(chunk * kAdamBlock) - (int64_t)(t.layout & 7u);
  if (base >= (int64_t)t.count) return;
  const uint32_t key = S8 ? mix32(s.key + (s.ordinal0 + (uint32_t)lo) * 0xB7E15163u) : 0;
  if ((t.layout & kAdamVec) && base >= 0 && base + kAdamBlock <= (int64_t)t.count)
    adamw_chunk<P, G, S8, true>(s, t, base, chunk, key, scale);
  else
    adamw_chunk<P, G, S8, false>(s, t, base, chunk, key, scale);
}

}  // namespace ra
