// One (parameter dtype, gradient dtype) slice of the AdamW kernels. The build
// compiles this file once per pair, with RA_SLICE_P and RA_SLICE_G set, so the
// nine slices compile in parallel; ra_adamw.cu dispatches to them.
#include "ra_adamw.cuh"

#if !defined(RA_SLICE_P) || !defined(RA_SLICE_G)
#error "compile with -DRA_SLICE_P=<dtype id> -DRA_SLICE_G=<dtype id>"
#endif

#define RA_CAT3_(a, b, c) a##_##b##_##c
#define RA_CAT3(a, b, c) RA_CAT3_(a, b, c)

namespace ra {
cudaError_t RA_CAT3(launch_adamw_small, RA_SLICE_P, RA_SLICE_G)(bool s8, const AdamArgs<kAdamSmall>& a, uint32_t ctas,
                                                                cudaStream_t s) {
  return s8 ? launch_programmatic(adamw_kernel<RA_SLICE_P, RA_SLICE_G, true, kAdamSmall>, dim3(ctas), kAdamThreads, 0, s, a)
            : launch_programmatic(adamw_kernel<RA_SLICE_P, RA_SLICE_G, false, kAdamSmall>, dim3(ctas), kAdamThreads, 0, s, a);
}
cudaError_t RA_CAT3(launch_adamw_large, RA_SLICE_P, RA_SLICE_G)(bool s8, const AdamArgs<kAdamLarge>& a, uint32_t ctas,
                                                                cudaStream_t s) {
  return s8 ? launch_programmatic(adamw_kernel<RA_SLICE_P, RA_SLICE_G, true, kAdamLarge>, dim3(ctas), kAdamThreads, 0, s, a)
            : launch_programmatic(adamw_kernel<RA_SLICE_P, RA_SLICE_G, false, kAdamLarge>, dim3(ctas), kAdamThreads, 0, s, a);
}
}  // namespace ra
