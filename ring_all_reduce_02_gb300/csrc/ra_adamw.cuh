// AdamW over many tensors in one launch, moments in fp32 or in 8 bits.
//
// Per element (g the scaled gradient, all fp32; in the moments every product and sum is rounded, the parameter's
// update is fused, with a reciprocal of a few ulp):
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// It touches every byte once: 4 + 4 + 2 + 8 + 8 + 2 = 28 bytes an element for
// fp32 parameters and moments with bf16 gradients and copies, 10 for bf16
// parameters with 8-bit moments.
//
// Work: a warp takes 256 consecutive elements (fp32 moments, 8 to a lane) or 512
// (8-bit, 16 to a lane: two blocks of the scales, each the share of half a warp),
// so that a block's largest magnitude is a few shuffles and the moments never
// leave registers between being read and being stored again. The tensors' table
// travels in the kernel's parameters. CTAs of 4 warps live for one such piece.
//
// Measured over 354.8 M elements in 292 tensors (back to back, inputs larger than
// L2): fp32 moments with bf16 gradients and copies 1394 us, 7.13 TB/s, 105% of the
// copy bandwidth: HBM is the bound. 8-bit moments on bf16 parameters 685 us, 5.2
// TB/s, 77% (without zeros among the second moments, see below): about 52 instructions an element (95 before pairs, Newton square
// roots and 16 elements a lane) take nearly as long as the memory, and the chain
// from the moments through the root, the block's maximum and the rounding is long
// for the 32 warps that the registers allow. 24 warps at 80 registers took 758 us,
// 40 warps with spills 719, 8 elements a lane 790 to 866; tiles prefetched into
// shared memory by resident warps 762.
#pragma once

#include <cuda_fp8.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"
#include "ra_tensors.cuh"

namespace ra {

constexpr int kAdamBlock = 256;  // elements per chunk, and per scale of an 8-bit moment
constexpr int kAdamThreads = 128;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamCtas = 8;  // on an SM: 64 registers a thread
// Consecutive elements of a lane.
__host__ __device__ constexpr int adam_lane_elems(bool s8) { return s8 ? 16 : 8; }
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
  uint32_t key;     // of its random bits
  uint32_t layout;  // kAdamVec: every buffer has vectors of 8 elements at elements 8 k - shift; low 3 bits: shift
};
constexpr uint32_t kAdamVec = 8;

// Kernel parameters hold at most 32,764 bytes. The small table shortens short lists' launches: 37 tensors take 45 us
// alone against 48 with the large one (the same 26 us back to back).
constexpr int kAdamSmall = 64;
constexpr int kAdamLarge = 384;

struct AdamScalars {
  float b1, one_minus_b1, b2, one_minus_b2, inv_sqrt_bc2, eps, step_size;
  float one;          // 1.0f, which the assembler must not know
  int n;              // tensors in the table
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

// A value scaled to its block (x * 448 / amax), rounded up or down by 16 random bits to the 3 bits that e4m3 keeps in
// its normal range: the bits below them decide with their own weight. The conversion that follows rounds what lies
// below that range once more, to nearest, and saturates, so that nothing passes 448.
__device__ __forceinline__ float round_up_or_down(float x, uint32_t rand16) {
  return __uint_as_float((__float_as_uint(x) + (rand16 << 4)) & 0xfff00000u);
}

// 8 consecutive elements as they are stored, and as fp32. The base is on the 8-element grid.
template <int DT>
using Raw8 = VecT<DT == DT_F32 ? 8 : 4>;
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* base, uint64_t i) {
  return ld_vec_w<DT == DT_F32 ? 8 : 4>(static_cast<const char*>(base) + i * Elem<DT>::kSize);
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& v, float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if constexpr (DT == DT_F32) f[k] = __uint_as_float(v.w[k]);
    else f[k] = widen16<DT>((v.w[k / 2] >> (k % 2 * 16)) & 0xffffu);
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
__device__ __forceinline__ uint2 load8_bytes(const void* base, uint64_t i) {
  return __ldcs(reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(base) + i));
}
__device__ __forceinline__ void widen8_e4m3(const uint2& q, float* f) {
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

// 1 / d to a few ulp (it only enters the parameter, where the step is a small part): d is sqrt(v) / sqrt(1 - b2^t)
// + eps with sqrt(v) either zero or above 2^-75, so it is no denormal unless eps is one.
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
// The largest magnitude and the largest value of three; a NaN wins the first and loses the second.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The negated square roots of two values -v from 2^-96 up, rounded to nearest: with y ~ 1/sqrt(v) and s = v y, the
// residual s^2 - v is exact in one fused operation and s - (s^2 - v) y/2 is Newton's next step, whose error is far
// below half an ulp (P. Markstein, IBM J. Res. Dev. 34, 1990). Equal to sqrtf for every significand. Signs are
// turned so that no operation is spent on them.
__device__ __forceinline__ F2 minus_sqrt2(F2 minus_v) {
  float v0, v1, y0, y1;
  split(minus_v, v0, v1);
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(-v0));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(-v1));
  const F2 y = pair(y0, y1), s = mul2(minus_v, y);
  return fma2(fma2(s, s, minus_v), mul2(y, twice(0.5f)), s);
}

// What a lane reads of whole chunks: its E consecutive elements.
template <int P, int G, bool S8, int E>
struct AdamRaw {
  Raw8<P> p[E / 8];
  Raw8<G> g[E / 8];
  Raw8<DT_F32> m[E / 8], v[E / 8];
};
template <int P, int G, int E>
struct AdamRaw<P, G, true, E> {
  Raw8<P> p[E / 8];
  Raw8<G> g[E / 8];
  uint2 m[E / 8], v[E / 8];
};

// A warp's elements base .. base + 32 E - 1 of a tensor, E to a lane. WHOLE: all of them exist and are on the
// 8-element grid of every buffer, and lane l takes base + E l .. base + E l + E - 1; a block of the 8-bit moments
// is then 256 / E lanes' share. Otherwise E = 8, only [0, count) exist, and lane l takes l, l + 32, ...
template <int P, int G, bool S8, bool WHOLE, int E>
__device__ __forceinline__ void adamw_elements(const AdamScalars& s, const AdamTensor& t, int64_t base, float scale) {
  static_assert(WHOLE || E == 8, "a whole share, or one block");
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t i0 = (uint64_t)base + (WHOLE ? E * lane : 0);
  const uint64_t block = S8 ? (WHOLE ? i0 : (uint64_t)base) / kAdamBlock : 0;  // 8-bit moments: base is on a block
  const auto at = [&](int j) { return WHOLE ? i0 + j : (uint64_t)(base + (int64_t)lane + 32 * j); };
  const auto in = [&](int j) { return WHOLE || at(j) < t.count; };  // a negative place wraps around
  float p[E], g[E], m[E], r[E];  // r: v; with 8-bit moments sqrt(v), and from then on its negative
  float m_scale = 0.0f, r_scale = 0.0f;
  if constexpr (WHOLE) {
    AdamRaw<P, G, S8, E> raw;
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      raw.g[k] = load8<G>(t.g, i0 + 8 * k);
      raw.p[k] = load8<P>(t.p, i0 + 8 * k);
      if constexpr (S8) raw.m[k] = load8_bytes(t.m, i0 + 8 * k), raw.v[k] = load8_bytes(t.v, i0 + 8 * k);
      else raw.m[k] = load8<DT_F32>(t.m, i0 + 8 * k), raw.v[k] = load8<DT_F32>(t.v, i0 + 8 * k);
    }
    if constexpr (S8) m_scale = t.ms[block], r_scale = t.vs[block];
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      widen8<G>(raw.g[k], g + 8 * k), widen8<P>(raw.p[k], p + 8 * k);
      if constexpr (S8) widen8_e4m3(raw.m[k], m + 8 * k), widen8_e4m3(raw.v[k], r + 8 * k);
      else widen8<DT_F32>(raw.m[k], m + 8 * k), widen8<DT_F32>(raw.v[k], r + 8 * k);
    }
  } else {
    if constexpr (S8) m_scale = t.ms[block], r_scale = t.vs[block];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      g[j] = in(j) ? load_as_f32<G>(t.g, at(j)) : 0.0f;
      p[j] = in(j) ? load_as_f32<P>(t.p, at(j)) : 0.0f;
      if constexpr (S8) m[j] = in(j) ? load_e4m3(t.m, at(j)) : 0.0f, r[j] = in(j) ? load_e4m3(t.v, at(j)) : 0.0f;
      else m[j] = in(j) ? load_as_f32<DT_F32>(t.m, at(j)) : 0.0f, r[j] = in(j) ? load_as_f32<DT_F32>(t.v, at(j)) : 0.0f;
    }
  }
  // the sign of the second moment's coefficients, see minus_sqrt2
  constexpr float kSign = S8 ? -1.0f : 1.0f;
  const F2 scale2 = twice(scale), b1 = twice(s.b1), b1c = twice(s.one_minus_b1);
  const F2 b2 = twice(kSign * s.b2), b2c = twice(kSign * s.one_minus_b2);
  const F2 one = twice(s.one), m_scale2 = twice(m_scale), r_scale2 = twice(r_scale);
  float most = -1.0f, r_top = 0.0f;
#pragma unroll
  for (int j = 0; j < E; j += 2) {
    const F2 gg = mul2(pair(g[j], g[j + 1]), scale2);
    F2 mm = pair(m[j], m[j + 1]), vv = pair(r[j], r[j + 1]);
    if constexpr (S8) mm = mul2(mm, m_scale2), vv = mul2(vv, r_scale2), vv = mul2(vv, vv);
    // Products and sums rounded one by one: the stored moments are the same bits as the formula's written out.
    // (x * 1 + y rather than x + y: the assembler contracts a mul.f32x2 and an add.f32x2, rounding modifiers or not.)
    mm = fma2(mul2(mm, b1), one, mul2(gg, b1c));
    vv = fma2(mul2(vv, b2), one, mul2(mul2(gg, b2c), gg));
    split(mm, m[j], m[j + 1]), split(vv, r[j], r[j + 1]);
    if constexpr (S8) {
      most = max3(most, r[j], r[j + 1]);
      split(minus_sqrt2(vv), r[j], r[j + 1]);
      r_top = max3_abs_nan(r_top, r[j], r[j + 1]);
    }
  }
  // zeros, values too small for minus_sqrt2, infinities: again by the book from what is in memory. One in a warp's
  // 512 elements is enough: with 2% of the gradients and moments zero, 354.8 M bf16 take 1560 us, not 685.
  bool plain = true;
  if constexpr (S8) {
    plain = most <= -0x1p-96f && r_top < __int_as_float(0x7f800000);
    if (!plain) {
      r_top = 0.0f;
#pragma unroll 1
      for (int k = 0; k < E; ++k) {
        float v = 0.0f;
        if (in(k)) {
          const float gk = load_as_f32<G>(t.g, at(k)) * scale, root = load_e4m3(t.v, at(k)) * r_scale;
          v = __fadd_rn(root * root * s.b2, gk * s.one_minus_b2 * gk);
        }
        v = __fsqrt_rn(v);
        r_top = fmaximum(r_top, v);
#pragma unroll
        for (int j = 0; j < E; ++j) r[j] = j == k ? -v : r[j];
      }
    }
  }
  const F2 bc = twice(kSign * s.inv_sqrt_bc2), eps = twice(s.eps), keep = twice(t.keep), step = twice(-s.step_size);
#pragma unroll
  for (int j = 0; j < E; j += 2) {
    const F2 root = S8 ? pair(r[j], r[j + 1]) : pair(__fsqrt_rn(r[j]), __fsqrt_rn(r[j + 1]));
    float d0, d1;
    split(fma2(root, bc, eps), d0, d1);
    const F2 u = mul2(pair(m[j], m[j + 1]), pair(reciprocal(d0), reciprocal(d1)));
    split(fma2(u, step, mul2(pair(p[j], p[j + 1]), keep)), p[j], p[j + 1]);
  }
  if constexpr (WHOLE) {
#pragma unroll
    for (int k = 0; k < E; k += 8) {
      store8<P>(t.p, i0 + k, p + k);
      if constexpr (!S8) store8<DT_F32>(t.m, i0 + k, m + k), store8<DT_F32>(t.v, i0 + k, r + k);
      if (t.copy != nullptr) {
        if (s.copy_dtype == DT_F32) store8<DT_F32>(t.copy, i0 + k, p + k);
        else if (s.copy_dtype == DT_F16) store8<DT_F16>(t.copy, i0 + k, p + k);
        else store8<DT_BF16>(t.copy, i0 + k, p + k);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
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
    float m_top = 0.0f;
#pragma unroll
    for (int j = 0; j < E; j += 2) m_top = max3_abs_nan(m_top, m[j], m[j + 1]);
    // the largest magnitudes of the block, as bits: they order as the values do, a NaN above infinity
    uint32_t m_bits = __float_as_uint(m_top), r_bits = __float_as_uint(r_top);
    constexpr int kLanes = 256 / E;  // of a block
    if constexpr (kLanes == 32) {
      m_bits = __reduce_max_sync(0xffffffffu, m_bits), r_bits = __reduce_max_sync(0xffffffffu, r_bits);
    } else {
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        m_bits = max(m_bits, __shfl_xor_sync(0xffffffffu, m_bits, o));
        r_bits = max(r_bits, __shfl_xor_sync(0xffffffffu, r_bits, o));
      }
    }
    const float m_amax = __uint_as_float(m_bits), r_amax = __uint_as_float(r_bits);
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);
    const bool m_some = m_amax > kMinAmax, r_some = r_amax > kMinAmax;
    const bool m_bad = !(m_amax < inf), r_bad = !(r_amax < inf);
    const float m_inv = m_some ? __frcp_rn(m_amax) * kE4m3Max : 0.0f;
    const float r_inv = r_some ? __frcp_rn(r_amax) * kE4m3Max : 0.0f;
    if (lane % kLanes == 0) {
      t.ms[block] = m_bad ? nan : m_some ? m_amax * (1.0f / kE4m3Max) : 0.0f;
      t.vs[block] = r_bad ? nan : r_some ? r_amax * (1.0f / kE4m3Max) : 0.0f;
    }
    const float r_floor = r_some ? 0.001953125f : 0.0f;  // 2^-9, the smallest value above zero
    const uint32_t seed0 = (uint32_t)i0 * 0x9E3779B9u + (uint32_t)(i0 >> 32) * 0xB7E15163u + t.key;
    const F2 m_inv2 = twice(m_inv), r_inv2 = twice(-r_inv);
    uint32_t zeros = 0;  // second moments that are
    if (!plain) {
#pragma unroll
      for (int j = 0; j < E; ++j) zeros |= (r[j] == 0.0f ? 1u : 0u) << j;
    }
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      split(mul2(pair(m[j], m[j + 1]), m_inv2), m[j], m[j + 1]);
      split(mul2(pair(r[j], r[j + 1]), r_inv2), r[j], r[j + 1]);
#pragma unroll
      for (int k = j; k < j + 2; ++k) {
        const uint64_t i = at(k);
        const uint32_t x = mix32_but_last(WHOLE ? seed0 + k * 0x9E3779B9u  // a lane's elements share i >> 32
                                                : (uint32_t)i * 0x9E3779B9u + (uint32_t)(i >> 32) * 0xB7E15163u + t.key);
        m[k] = round_up_or_down(m[k], (x ^ (x >> 16)) & 0xffffu);
        r[k] = fmaxf(round_up_or_down(r[k], x >> 16), r_floor);
      }
    }
    if (!plain) {
#pragma unroll
      for (int j = 0; j < E; ++j) r[j] = zeros >> j & 1u ? 0.0f : r[j];
    }
    if constexpr (WHOLE) {
      uint32_t mq[E / 4], rq[E / 4];
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        mq[k] = m_bad ? 0x7f7f7f7fu : pack4_e4m3(m + 4 * k);
        rq[k] = r_bad ? 0x7f7f7f7fu : pack4_e4m3(r + 4 * k);
      }
      unsigned char *to_m = static_cast<unsigned char*>(t.m) + i0, *to_r = static_cast<unsigned char*>(t.v) + i0;
#pragma unroll
      for (int k = 0; k < E / 4; k += 2) {
        __stcs(reinterpret_cast<uint2*>(to_m + 4 * k), make_uint2(mq[k], mq[k + 1]));
        __stcs(reinterpret_cast<uint2*>(to_r + 4 * k), make_uint2(rq[k], rq[k + 1]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if (!in(j)) continue;
        static_cast<unsigned char*>(t.m)[at(j)] = m_bad ? 0x7f : __nv_cvt_float_to_fp8(m[j], __NV_SATFINITE, __NV_E4M3);
        static_cast<unsigned char*>(t.v)[at(j)] = r_bad ? 0x7f : __nv_cvt_float_to_fp8(r[j], __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

template <int P, int G, bool S8, int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas) adamw_kernel(const __grid_constant__ AdamArgs<CAP> a) {
  pdl_enter();
  const AdamScalars& s = a.s;
  float scale = 1.0f;
  if (s.scale != nullptr) {
    scale = *s.scale;
    if (!(fabsf(scale) < __int_as_float(0x7f800000))) return;  // not finite: the step is skipped
  }
  const int lo = last_not_above(a.cta0, s.n, blockIdx.x);
  const AdamTensor& t = a.t[lo];
  constexpr int E = adam_lane_elems(S8);
  const uint64_t warp = (uint64_t)(blockIdx.x - a.cta0[lo]) * kAdamWarps + threadIdx.x / 32;
  int64_t base = (int64_t)(warp * (32 * E)) - (int64_t)(t.layout & 7u);
  const int64_t count = (int64_t)t.count;
  if ((t.layout & kAdamVec) && base >= 0 && base + 32 * E <= count) {
    adamw_elements<P, G, S8, true, E>(s, t, base, scale);
  } else {
#pragma unroll 1
    for (int k = 0; k < E / 8 && base < count; ++k, base += kAdamBlock) {
      // a tensor's end: its last whole block still goes in vectors (59 odd-sized tensors, 1.9 M elements: 12.3 -> 10.9 us)
      if (S8 && (t.layout & kAdamVec) && base + kAdamBlock <= count) adamw_elements<P, G, S8, true, 8>(s, t, base, scale);
      else adamw_elements<P, G, S8, false, 8>(s, t, base, scale);
    }
  }
}

}  // namespace ra
