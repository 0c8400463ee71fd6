// One (row dtype, weight dtype) slice of the layer norm kernels and their launch
// shapes. The build compiles this file once per pair, with RA_SLICE_DT and
// RA_SLICE_W set, so the five slices compile in parallel.
#include "ra_layernorm.cuh"

#if !defined(RA_SLICE_DT) || !defined(RA_SLICE_W)
#error "compile with -DRA_SLICE_DT=<dtype id> -DRA_SLICE_W=<dtype id>"
#endif

#define RA_CAT3_(a, b, c) a##_##b##_##c
#define RA_CAT3(a, b, c) RA_CAT3_(a, b, c)

namespace ra {
namespace {

constexpr int DT = RA_SLICE_DT, WDT = RA_SLICE_W;
constexpr uint32_t es = Elem<DT>::kSize;

constexpr uint32_t V = 16 / es;
constexpr size_t kLnSmem = 226 * 1024;  // dynamic shared memory a CTA may take

uint32_t phase(const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u); }
uint32_t line(uint64_t stride) { return (uint32_t)(stride * es & 15u); }
unsigned row_ctas(uint64_t rows) { return (unsigned)(rows < 152 * 8 ? rows : 152 * 8); }

// Threads per row: the fewest that hold it in `per` columns each.
uint32_t group_for(uint64_t cols, uint64_t per, uint32_t least, uint32_t most) {
  uint32_t group = least;
  while (group < most && group * per < cols) group *= 2;
  return group;
}

template <class K>
cudaError_t allow_smem(K kernel, size_t smem) {
  return smem <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <int E>
cudaError_t forward_registers(const LnForward& a, uint32_t group, cudaStream_t s) {
  const uint64_t per_cta = group == 32 ? kLnWarpThreads / 32 : 1, ctas = (a.rows + per_cta - 1) / per_cta;
  if (ctas > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  return group == 32 ? launch_programmatic(ln_forward_registers<DT, WDT, E, true>, dim3((unsigned)ctas), kLnWarpThreads, 0, s, a)
                     : launch_programmatic(ln_forward_registers<DT, WDT, E, false>, dim3((unsigned)ctas), group, 0, s, a);
}
template <int E>
cudaError_t forward_shifted(const LnForward& a, uint32_t group, size_t smem, cudaStream_t s) {
  const cudaError_t err = allow_smem(ln_forward_shifted<DT, WDT, E>, smem);
  if (err != cudaSuccess) return err;
  uint64_t per_sm = 1024 / group;
  if (per_sm > kLnSmem / (smem + 1280)) per_sm = kLnSmem / (smem + 1280);
  if (per_sm < 1) per_sm = 1;
  const uint64_t ctas = a.rows < 152 * per_sm ? a.rows : 152 * per_sm;
  return launch_programmatic(ln_forward_shifted<DT, WDT, E>, dim3((unsigned)ctas), group, smem, s, a);
}

template <int E>
cudaError_t backward_fused(const LnBackward& a, bool shifted, size_t smem, cudaStream_t s) {
  const auto kernel = shifted ? ln_backward_fused<DT, WDT, E, true> : ln_backward_fused<DT, WDT, E, false>;
  const cudaError_t err = allow_smem(kernel, smem);
  return err != cudaSuccess ? err : launch_programmatic(kernel, dim3((unsigned)a.parts), kLnMaxThreads, smem, s, a);
}

}  // namespace

cudaError_t RA_CAT3(ln_forward, RA_SLICE_DT, RA_SLICE_W)(const LnForward& a, cudaStream_t s) {
  const bool aligned = a.cols % V == 0 && !phase(a.x) && !phase(a.y) && !line(a.x_stride) && !line(a.y_stride) &&
                       !phase(a.w) && !phase(a.b);
  if (aligned && a.cols <= (uint64_t)kLnMaxThreads * 64) {
    const uint32_t group = group_for(a.cols, 32, 32, kLnMaxThreads);
    const uint64_t per = (a.cols + group - 1) / group;
    if (per <= 8) return forward_registers<8>(a, group, s);
    if (per <= 16) return forward_registers<16>(a, group, s);
    if (per <= 24) return forward_registers<24>(a, group, s);
    if (per <= 32) return forward_registers<32>(a, group, s);
    return forward_registers<64>(a, group, s);
  }
  // x and y in step: every row of both at the same place in its 16-byte line
  if (phase(a.x) == phase(a.y) && line(a.x_stride) == line(a.y_stride) && a.cols < 1u << 20) {
    const uint64_t cols = a.cols + V - 1;  // a line more, at most
    const size_t smem = gapped_size<V>((uint32_t)a.cols) * sizeof(float2);
    const uint32_t group = group_for(cols, 16, 64, kLnMaxThreads);
    const uint64_t per = (cols + group - 1) / group;
    if (smem <= kLnSmem && per <= 64) {
      if (per <= 8) return forward_shifted<8>(a, group, smem, s);
      if (per <= 16) return forward_shifted<16>(a, group, smem, s);
      if (per <= 32) return forward_shifted<32>(a, group, smem, s);
      return forward_shifted<64>(a, group, smem, s);
    }
  }
  return launch_programmatic(ln_forward_rows<DT, WDT>, dim3(row_ctas(a.rows)), kLnThreads, 0, s, a);
}

cudaError_t RA_CAT3(ln_backward, RA_SLICE_DT, RA_SLICE_W)(LnBackward a, cudaStream_t s) {
  const bool sums = a.dw != nullptr || a.db != nullptr;
  const unsigned slices = (unsigned)((a.cols + 31) / 32);
  cudaError_t err;
  const bool aligned = a.cols % V == 0 && !phase(a.x) && !phase(a.dy) && !phase(a.dx) && !line(a.x_stride) &&
                       !line(a.dy_stride) && !line(a.dx_stride);
  const bool in_step = phase(a.x) == phase(a.dy) && phase(a.x) == phase(a.dx) && line(a.x_stride) == line(a.dy_stride) &&
                       line(a.x_stride) == line(a.dx_stride);
  const uint64_t reach = a.cols + (aligned ? 0 : V - 1);
  // the sweep in one kernel wants a row in 32 columns a thread and two rows of x and dy per group in shared memory
  if (a.rows > 0 && in_step && reach <= (uint64_t)kLnMaxThreads * 32) {
    const uint32_t cols = (uint32_t)a.cols;
    const size_t fixed = ln_weight_bytes(cols, es, !aligned), row = 2 * ln_row_bytes(cols, es, !aligned);
    a.group = group_for(reach, 32, 32, kLnMaxThreads);
    uint32_t groups = kLnMaxThreads / a.group;
    size_t stages = (kLnSmem - fixed) / (groups * row);
    while (stages < 2 && a.group < kLnMaxThreads) {
      a.group *= 2, groups /= 2;
      stages = (kLnSmem - fixed) / (groups * row);
    }
    if (stages >= 2) {
      a.stages = stages > 4 ? 4 : (uint32_t)stages;
      size_t smem = fixed + groups * a.stages * row;
      const size_t fold = (size_t)groups * 2 * cols * 4;
      if (fold > smem) smem = fold;
      const uint64_t per = (reach + a.group - 1) / a.group;
      if (per <= 8) err = backward_fused<8>(a, !aligned, smem, s);
      else if (per <= 16) err = backward_fused<16>(a, !aligned, smem, s);
      else if (per <= 24) err = backward_fused<24>(a, !aligned, smem, s);
      else err = backward_fused<32>(a, !aligned, smem, s);
      if (err != cudaSuccess || !sums) return err;
      return launch_programmatic(ln_backward_finish<WDT>, dim3(slices), kLnFinishThreads, 0, s, a);
    }
  }
  if (sums) {  // before dx, which may be x or dy
    if (a.parts) {
      err = launch_programmatic(ln_backward_columns<DT>, dim3(slices, (unsigned)a.parts), kLnThreads, 0, s, a);
      if (err != cudaSuccess) return err;
    }
    err = launch_programmatic(ln_backward_finish<WDT>, dim3(slices), kLnFinishThreads, 0, s, a);
    if (err != cudaSuccess) return err;
  }
  if (a.rows == 0) return cudaSuccess;
  return launch_programmatic(ln_backward_rows<DT, WDT>, dim3(row_ctas(a.rows)), kLnThreads, 0, s, a);
}

}  // namespace ra
