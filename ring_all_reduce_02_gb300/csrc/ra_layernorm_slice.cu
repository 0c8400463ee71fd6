// One (row dtype, weight dtype) slice of the layer norm kernels and their launch
// shapes. The build compiles this file once per pair, with RA_SLICE_DT and
// RA_SLICE_W set, so the five slices compile in parallel.
#include <type_traits>

#include "ra_layernorm.cuh"
#include "ra_layernorm_plan.h"

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

// Threads for a row of `cols` columns, `per` or fewer to each: whole warps.
uint32_t group_for(uint64_t cols, uint32_t per) { return (uint32_t)((cols + 32 * per - 1) / (32 * per)) * 32; }

// Lets a kernel take `smem` bytes. The limit is the function's, not the call's: it is set to the same value by every
// call, so that none of another thread's lowers it between this and the launch.
template <class K>
cudaError_t allow_smem(K kernel, size_t smem) {
  if (smem <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLnSmem);
}

// launch(std::bool_constant): the kernel with a second mean or without, as rows of `cols` columns (LEAST to MOST) have it.
template <uint64_t LEAST, uint64_t MOST, class F>
cudaError_t with_second(uint64_t cols, F launch) {
  constexpr bool never = DT == DT_BF16 || (DT == DT_F16 && MOST <= 8192), always = DT == DT_F32 || (DT == DT_F16 && LEAST > 8192);
  if constexpr (never) return launch(std::false_type{});
  else if constexpr (always) return launch(std::true_type{});
  else return second_mean<DT>(cols) ? launch(std::true_type{}) : launch(std::false_type{});
}

// E columns a thread: a row to each warp of a CTA, or rows of LEAST columns or more to a CTA of `group` threads.
template <int E>
cudaError_t forward_warps(const LnForward& a, cudaStream_t s) {
  constexpr uint64_t per_cta = kLnWarpThreads / 32;
  return with_second<0, E * 32>(a.cols, [&](auto second) {
    return launch_programmatic(ln_forward_registers<DT, WDT, E, true, decltype(second)::value>,
                               dim3((unsigned)((a.rows + per_cta - 1) / per_cta)), kLnWarpThreads, 0, s, a);
  });
}
template <int E, uint64_t LEAST>
cudaError_t forward_registers(const LnForward& a, uint32_t group, cudaStream_t s) {
  return with_second<LEAST, E * kLnMaxThreads>(a.cols, [&](auto second) {
    return launch_programmatic(ln_forward_registers<DT, WDT, E, false, decltype(second)::value>, dim3((unsigned)a.rows), group, 0, s,
                               a);
  });
}
// CTAs, each with a row of `reach` columns, that an SM holds at `per` columns a thread: by registers (64, 85 or 128 a
// thread) and by the shared memory for the weights.
uint64_t shifted_rows(uint64_t reach, uint32_t per, size_t smem) {
  const uint64_t by_registers = (per <= 16 ? 1024 : per == 24 ? 768 : 512) / group_for(reach, per);
  const uint64_t by_smem = kLnSmem / (smem + 1280);
  const uint64_t rows = by_registers < by_smem ? by_registers : by_smem;
  return rows < 1 ? 1 : rows;
}

template <int E, uint64_t LEAST>
cudaError_t forward_shifted(const LnForward& a, uint32_t group, size_t smem, cudaStream_t s) {
  return with_second<LEAST, E * kLnMaxThreads>(a.cols, [&](auto second) {
    const auto kernel = ln_forward_shifted<DT, WDT, E, decltype(second)::value>;
    const cudaError_t err = allow_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    const uint64_t per_sm = shifted_rows((uint64_t)group * E, E, smem);
    const uint64_t ctas = a.rows < 152 * per_sm ? a.rows : 152 * per_sm;
    return launch_programmatic(kernel, dim3((unsigned)ctas), group, smem, s, a);
  });
}

template <int E, bool KEEP>
cudaError_t backward_fused(LnBackward* all, bool shifted, size_t weights, size_t stage, cudaStream_t s) {
  LnBackward& a = *all;
  const uint32_t groups = kLnMaxThreads / a.group;
  // up to two rows a group are one CTA's: a second round costs less than the launch that would add the partials. Not
  // off the 16-byte grid, where the rows of a CTA have to be a multiple of 8 apart to share a phase.
  if (!shifted && a.rows <= 2 * groups) a.parts = 1;
  const size_t stages = (kLnSmem - weights) / (groups * stage);
  a.stages = stages >= 8 ? 8 : stages >= 6 ? 6 : stages >= 4 ? 4 : (uint32_t)stages;
  size_t smem = weights + groups * a.stages * stage;
  if (smem < groups * 2 * weights) smem = groups * 2 * weights;  // the fold
  const auto kernel = shifted ? ln_backward_fused<DT, WDT, E, KEEP, true, false>
                              : ln_backward_fused<DT, WDT, E, KEEP, false, false>;
  const cudaError_t err = allow_smem(kernel, smem);
  return err != cudaSuccess ? err : launch_programmatic(kernel, dim3((unsigned)a.parts), groups * a.group, smem, s, a);
}

// The fused kernel with a cluster of a.split CTAs to a row; a.parts becomes the number of clusters. Where the device
// holds too few (it may be shared out), nothing is launched and *fits becomes false.
template <int E>
cudaError_t backward_late(LnBackward* a, bool shifted, size_t weights, size_t stage, cudaStream_t s, bool* fits) {
  const size_t stages = (kLnSmem - weights) / stage;
  a->stages = stages >= 8 ? 8 : stages >= 6 ? 6 : stages >= 4 ? 4 : (uint32_t)stages;
  size_t smem = weights + a->stages * stage;
  if (smem < 2 * weights) smem = 2 * weights;  // the fold
  const auto kernel = shifted ? ln_backward_fused<DT, WDT, E, false, true, true>
                              : ln_backward_fused<DT, WDT, E, false, false, true>;
  cudaError_t err = allow_smem(kernel, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a->split, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kLnMaxParts / a->split * a->split));
  cfg.blockDim = dim3(a->group);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  err = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
  if (err != cudaSuccess) return err;
  if (clusters > (int)(kLnMaxParts / a->split)) clusters = (int)(kLnMaxParts / a->split);
  const uint64_t parts = late_clusters((uint64_t)clusters, a->rows, shifted ? V : 1);
  *fits = parts > 0;
  if (!*fits) return cudaSuccess;
  a->parts = (int)parts;
  cfg.gridDim = dim3((unsigned)a->parts * a->split);
  cfg.numAttrs = RA_PDL ? 2 : 1;
  err = cudaLaunchKernelEx(&cfg, kernel, *a);
  const cudaError_t last = cudaGetLastError();
  return err != cudaSuccess ? err : last;
}

}  // namespace

cudaError_t RA_CAT3(ln_forward, RA_SLICE_DT, RA_SLICE_W)(const LnForward& a, cudaStream_t s) {
  const bool aligned = a.cols % V == 0 && !phase(a.x) && !phase(a.y) && !line(a.x_stride) && !line(a.y_stride) &&
                       !phase(a.w) && !phase(a.b);
  if (aligned && a.cols <= (uint64_t)kLnMaxThreads * 64 && a.rows <= 0x7fffffffull) {  // a CTA for every row, or for 4
    if (a.cols <= 256) return forward_warps<8>(a, s);
    if (a.cols <= 512) return forward_warps<16>(a, s);
    // few rows leave SMs idle: more threads to a row, fewer columns each (1 x 1024: 1.6 us against 2.1, 512 x 1024: 2.4
    // against 2.8); many rows want the row's fixed cost on few threads (8192 x 4096: 24 us against 36)
    if (a.rows <= 608 && a.cols <= 4096) return forward_registers<8, 513>(a, group_for(a.cols, 8), s);
    if (a.cols <= 1024) return forward_warps<32>(a, s);
    if (a.cols <= 16384) return forward_registers<32, 1025>(a, group_for(a.cols, 32), s);
    return forward_registers<64, 16385>(a, group_for(a.cols, 64), s);
  }
  // x and y in step: every row of both at the same place in its 16-byte line
  const uint64_t reach = a.cols + V - 1;  // a line more, at most
  if (phase(a.x) == phase(a.y) && line(a.x_stride) == line(a.y_stride) && reach <= (uint64_t)kLnMaxThreads * 64) {
    const size_t smem = 2 * sizeof(float) * ln_share_elems((uint32_t)a.cols, es, true, 1);
    if (smem <= kLnSmem) {
      if (reach > 8192 && reach <= 9216) return forward_shifted<24, 0>(a, group_for(reach, 24), smem, s);
      if (reach <= 8192) {
        // More columns a thread leave fewer warps that are partly empty. Taken where a third more rows are at work on
        // an SM and there are rows enough for the longer start: 16000 x 4095 bf16 58.4 -> 51.0 us, 16000 x 701 19.2 ->
        // 14.7, but 1200 x 701 4.9 -> 6.0; with a fifth more rows, 16000 x 1201 21.7 -> 22.7.
        const bool wider = a.rows > 4096 && 3 * shifted_rows(reach, reach <= 512 ? 16 : 24, smem) >=
                                                4 * shifted_rows(reach, reach <= 512 ? 8 : 16, smem);
        if (reach <= 512) {
          return wider ? forward_shifted<16, 0>(a, group_for(reach, 16), smem, s)
                       : forward_shifted<8, 0>(a, group_for(reach, 8), smem, s);
        }
        return wider ? forward_shifted<24, 0>(a, group_for(reach, 24), smem, s)
                     : forward_shifted<16, 0>(a, group_for(reach, 16), smem, s);
      }
      if (reach <= 16384) return forward_shifted<32, 9217 - V>(a, group_for(reach, 32), smem, s);
      // 64 columns a thread spill; at 4 bytes a column the general kernel is faster (3000 x 23001 fp32, one mean: 230 us, not 405)
      if constexpr (es == 2) return forward_shifted<64, 16385 - V>(a, group_for(reach, 64), smem, s);
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
  // the sweep in one kernel: two stages of a row's x and dy for each group have to fit in shared memory
  const auto finish = [&]() {
    if (!sums || a.parts == 1) return cudaSuccess;
    return launch_programmatic(ln_backward_finish<WDT>, dim3(slices), kLnFinishThreads, 0, s, a);
  };
  if (a.rows > 0 && in_step && reach <= (uint64_t)kLnMaxThreads * 32) {
    const uint32_t elems = ln_share_elems((uint32_t)a.cols, es, !aligned, 1);
    const size_t weights = elems * 4, row = 2 * elems * es;
    // 16 columns a thread keep xhat and dy w in registers; 24 and 32 take them from shared memory again and are
    // worth about 0.8 and 0.5 of a thread of 16, but win where they put more of the CTA's 512 threads to work (a
    // group is whole warps): 4096 x 5120 fp32 and 4096 x 6001 bf16 take 9% less with 24 than with 16,
    // 6001 x 4095 fp16 13% (19% less than with 32)
    const auto score = [&](uint32_t per) {
      const uint32_t group = group_for(reach, per), groups = group ? kLnMaxThreads / group : 0;
      if (groups == 0 || weights + 2 * groups * row > kLnSmem) return 0.0;
      return groups * group * (per == 16 ? 1.0 : per == 24 ? 0.8 : 0.5);
    };
    const double s16 = score(16), s24 = score(24), s32 = es == 2 ? score(32) : 0.0;  // of 4 bytes it is never the best
    const uint32_t per = reach <= 256 ? 8 : s16 >= s24 && s16 >= s32 ? 16 : s24 >= s32 ? 24 : 32;
    if (s16 + s24 + s32 > 0.0) {
      a.group = group_for(reach, per);
      if (per == 8) err = backward_fused<8, true>(&a, !aligned, weights, row, s);
      else if (per == 16) err = backward_fused<16, true>(&a, !aligned, weights, row, s);
      else if (es == 4 || per == 24) err = backward_fused<24, false>(&a, !aligned, weights, row, s);
      else if constexpr (es == 2) err = backward_fused<32, false>(&a, !aligned, weights, row, s);
      return err != cudaSuccess ? err : finish();
    }
  }
  // else a row shared by the fewest CTAs that hold it (where one CTA does, sharing takes longer: half as long again
  // at 4096 x 12288 bf16, 30% at 4096 x 10000 fp32)
  for (uint32_t split = 2; a.rows > 0 && in_step && split <= kLnMaxSplit; split *= 2) {
    if (a.cols > (uint64_t)kLnMaxThreads * 24 * split) continue;
    const uint32_t share = ln_share_elems((uint32_t)a.cols, es, !aligned, split), per = share <= kLnMaxThreads * 16 ? 16 : 24;
    const size_t weights = share * 4, row = 2 * share * es;
    if (share > kLnMaxThreads * per || weights + 2 * row > kLnSmem) continue;
    a.split = split;
    a.group = group_for(share, per);
    bool fits = true;
    err = per == 16 ? backward_late<16>(&a, !aligned, weights, row, s, &fits)
                    : backward_late<24>(&a, !aligned, weights, row, s, &fits);
    if (err != cudaSuccess || fits) return err != cudaSuccess ? err : finish();
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
