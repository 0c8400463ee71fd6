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

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool rows16(const void* p, uint64_t stride) { return on16(p) && stride * es % 16 == 0; }
unsigned row_ctas(uint64_t rows) { return (unsigned)(rows < 152 * 8 ? rows : 152 * 8); }

// Threads per row: the fewest that hold it in 32 columns each.
uint32_t group_for(uint64_t cols, uint32_t most) {
  uint32_t group = 32;
  while (group < most && (uint64_t)group * 32 < cols) group *= 2;
  return group;
}

template <int E>
cudaError_t forward_registers(const LnForward& a, bool vector, cudaStream_t s) {
  const uint32_t threads = a.group > 128 ? a.group : 128;
  const uint64_t ctas = (a.rows + threads / a.group - 1) / (threads / a.group);
  if (ctas > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  return vector ? launch_programmatic(ln_forward_registers<DT, WDT, E, true>, dim3((unsigned)ctas), threads, 0, s, a)
                : launch_programmatic(ln_forward_registers<DT, WDT, E, false>, dim3((unsigned)ctas), threads, 0, s, a);
}

template <int E>
cudaError_t backward_fused(const LnBackward& a, bool vector, size_t smem, cudaStream_t s) {
  const auto kernel = vector ? ln_backward_fused<DT, WDT, E, true> : ln_backward_fused<DT, WDT, E, false>;
  if (smem > 48 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  return launch_programmatic(kernel, dim3((unsigned)a.parts), kLnMaxThreads, smem, s, a);
}

}  // namespace

cudaError_t RA_CAT3(ln_forward, RA_SLICE_DT, RA_SLICE_W)(LnForward a, cudaStream_t s) {
  if (a.cols > (uint64_t)kLnMaxThreads * 64)
    return launch_programmatic(ln_forward_rows<DT, WDT>, dim3(row_ctas(a.rows)), kLnThreads, 0, s, a);
  const bool vector = a.cols * es % 16 == 0 && rows16(a.x, a.x_stride) && rows16(a.y, a.y_stride) && on16(a.w) && on16(a.b);
  a.group = group_for(a.cols, kLnMaxThreads);
  const uint64_t per = (a.cols + a.group - 1) / a.group;
  if (per <= 8) return forward_registers<8>(a, vector, s);
  if (per <= 16) return forward_registers<16>(a, vector, s);
  if (per <= 24) return forward_registers<24>(a, vector, s);
  if (per <= 32) return forward_registers<32>(a, vector, s);
  return forward_registers<64>(a, vector, s);
}

cudaError_t RA_CAT3(ln_backward, RA_SLICE_DT, RA_SLICE_W)(LnBackward a, cudaStream_t s) {
  const bool sums = a.dw != nullptr || a.db != nullptr;
  const unsigned slices = (unsigned)((a.cols + 31) / 32);
  cudaError_t err;
  // the sweep in one kernel wants a row in 32 columns a thread and two rows of x and dy per group in shared memory
  if (a.rows > 0 && a.cols <= (uint64_t)kLnMaxThreads * 32) {
    const bool vector = a.cols * es % 16 == 0 && rows16(a.x, a.x_stride) && rows16(a.dy, a.dy_stride) && rows16(a.dx, a.dx_stride);
    const uint32_t cols = (uint32_t)a.cols;
    const size_t limit = 226 * 1024, fixed = (cols * 4 + 15) / 16 * 16, row = 2 * ln_row_bytes(cols, es, vector);
    a.group = group_for(cols, kLnMaxThreads);
    uint32_t groups = kLnMaxThreads / a.group;
    size_t stages = (limit - fixed) / (groups * row);
    while (stages < 2 && a.group < kLnMaxThreads) {
      a.group *= 2, groups /= 2;
      stages = (limit - fixed) / (groups * row);
    }
    if (stages >= 2) {
      a.stages = stages > 4 ? 4 : (uint32_t)stages;
      size_t smem = fixed + groups * a.stages * row;
      const size_t fold = (size_t)groups * 2 * cols * 4;
      if (fold > smem) smem = fold;
      const uint64_t per = (cols + a.group - 1) / a.group;
      if (per <= 8) err = backward_fused<8>(a, vector, smem, s);
      else if (per <= 16) err = backward_fused<16>(a, vector, smem, s);
      else if (per <= 24) err = backward_fused<24>(a, vector, smem, s);
      else err = backward_fused<32>(a, vector, smem, s);
      if (err != cudaSuccess || !sums) return err;
      return launch_programmatic(ln_backward_finish<WDT>, dim3(slices), kLnThreads, 0, s, a);
    }
  }
  if (sums) {  // before dx, which may be x or dy
    if (a.parts) {
      err = launch_programmatic(ln_backward_columns<DT>, dim3(slices, (unsigned)a.parts), kLnThreads, 0, s, a);
      if (err != cudaSuccess) return err;
    }
    err = launch_programmatic(ln_backward_finish<WDT>, dim3(slices), kLnThreads, 0, s, a);
    if (err != cudaSuccess) return err;
  }
  if (a.rows == 0) return cudaSuccess;
  return launch_programmatic(ln_backward_rows<DT, WDT>, dim3(row_ctas(a.rows)), kLnThreads, 0, s, a);
}

}  // namespace ra
