// Pairs of fp32: sm_103a adds, multiplies and fuses two fp32 in one instruction,
// each rounded as the scalar operation is. At 4 to 10 bytes of HBM traffic per
// element an SM has 23 to 55 issue slots per element, so pairs are what keeps the
// layer norm and 8-bit AdamW kernels near the memory's rate.
#pragma once

#include <stdint.h>

namespace ra {

using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(F2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 twice(float a) { return pair(a, a); }
__device__ __forceinline__ float fold2(F2 p) {
  float a, b;
  split(p, a, b);
  return a + b;
}

}  // namespace ra
