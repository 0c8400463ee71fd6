// ra_cross_entropy_forward / _backward: argument checks, scratch, launches.
#include <cudaTypedefs.h>
#include <math.h>

#include "ra_cross_entropy.cuh"
#include "ra_cross_entropy_plan.h"
#include "ra_host.h"

namespace {

using ra::Buffer;
using ra::CeArgs;
using ra::CePlan;

constexpr uint64_t kMostRows = (1ull << 31) - 1024;
// A tile of logits sums over all columns, by one pair of CTAs: 2^18 blocks take it under a second, and no wait for it
// comes near its limit.
constexpr uint64_t kMostCols = 1ull << 24;

unsigned at_most(uint64_t n, uint64_t most) { return (unsigned)(n < most ? n : most); }

bool in_place(const void* weight, uint64_t stride) {
  return reinterpret_cast<uintptr_t>(weight) % 16 == 0 && stride % 8 == 0 && stride < 1ull << 38;
}

bool sizes_ok(uint64_t rows, uint64_t cols, uint64_t vocab) {
  return rows <= kMostRows && vocab <= kMostRows && cols <= kMostCols && ra::shape_ok(rows, cols) && ra::shape_ok(vocab, cols);
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t s, A... args) {
  return ra::launch_programmatic(kernel, grid, threads, 0, s, args...);
}

// The rows that count, and the operands in the form that the products take.
template <bool BACKWARD>
cudaError_t rows_and_operands(const CeArgs& a, cudaStream_t s) {
  cudaError_t err = launch(ra::ce_rows_kernel<BACKWARD>, dim3((unsigned)a.parts), ra::kCeRowsThreads, s, a);
  if (err == cudaSuccess && a.w != a.weight) err = launch(ra::ce_weight_kernel, dim3(at_most((a.vocab + 7) / 8, 152 * 8)), 256, s, a);
  return err;
}

// Tensor maps of a [rows][cols] matrix of 16-bit elements with swizzled rows of 64: in boxes of 64 columns and `high`
// rows, or (groups) of 64 rows and two groups of 64 columns, one behind the other. Columns are whole groups then.
cudaError_t encode(CUtensorMap* map, int dtype, const void* p, uint64_t cols, uint64_t rows, uint64_t stride, uint32_t high,
                   bool groups = false) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    return err == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  if (fn == nullptr) return cudaErrorInitializationError;
  const cuuint64_t size[3] = {groups ? 64 : cols, rows, cols / 64}, strides[2] = {stride * 2, 128};
  const cuuint32_t box[3] = {64, high, 2}, steps[3] = {1, 1, 1};
  const CUresult r = fn(map, dtype == RA_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 3 : 2,
                        const_cast<void*>(p), size, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// The maps of both passes.
cudaError_t encode_logits(ra::CeTiles& t, int dtype) {
  const CeArgs& a = t.a;
  const cudaError_t err = encode(&t.h, dtype, a.h, a.cols_pad, a.rows_pad, a.cols_pad, a.rows <= ra::kCeFew ? 64 : 128);
  return err != cudaSuccess ? err : encode(&t.w, dtype, a.w, a.cols, a.vocab, a.w_stride, (uint32_t)a.words / 2);
}

// Every SM has a CTA at most; all rows are taken to count.
template <int DT, int WDT, bool BACKWARD, bool CHUNKS>
cudaError_t launch_tiles(const ra::CeTiles& t, uint64_t tiles, cudaStream_t s) {
  const auto kernel = ra::ce_tiles_kernel<DT, WDT, BACKWARD, CHUNKS>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ra::kCeSmem);
  return err != cudaSuccess ? err
                            : ra::launch_programmatic(kernel, dim3(2 * at_most(tiles, ra::kCePairs)), ra::kCeThreads, ra::kCeSmem, s, t);
}

// How long a wait inside a kernel may take, and what the self-test withholds from it.
struct Limits {
  uint64_t wait_ns = ra::kPairWaitNs;
  int withheld = ra::CE_NOTHING;
};

template <int DT>
cudaError_t forward(const CeArgs& a, const Limits& limits, cudaStream_t s) {
  ra::CeTiles t = {};
  t.a = a, t.w_out = a.vocab, t.counter = a.counters, t.wait_ns = limits.wait_ns, t.withheld = limits.withheld;
  cudaError_t err = encode_logits(t, DT);
  if (err == cudaSuccess) err = rows_and_operands<false>(a, s);
  t.early = a.rows <= ra::kCeFew && a.w == a.weight;
  if (err == cudaSuccess) err = launch_tiles<DT, DT, false, true>(t, a.rows_pad / 256 * (a.slots / 2), s);
  if (err != cudaSuccess) return err;
  // few rows: a CTA to each
  return a.rows <= 512 ? launch(ra::ce_join_kernel<8>, dim3((unsigned)a.rows), 256, s, a)
                       : launch(ra::ce_join_kernel<1>, dim3((unsigned)((a.rows + 7) / 8)), 256, s, a);
}

template <int DT, int WDT>
cudaError_t backward(const CeArgs& a, const CePlan& p, char* scratch, const Limits& limits, cudaStream_t s) {
  ra::CeTiles t = {};
  t.a = a, t.wait_ns = limits.wait_ns, t.withheld = limits.withheld;
  CUtensorMap g[2], g_own[2], g_store[2];
  t.w_groups = a.w != a.weight || a.cols % 64 == 0;
  cudaError_t err = encode_logits(t, DT);
  if (err == cudaSuccess) err = encode(&t.h_own, DT, a.h, a.cols_pad, a.rows_pad, a.cols_pad, 64, true);
  if (err == cudaSuccess)
    err = t.w_groups ? encode(&t.w_own, DT, a.w, (a.cols + 63) / 64 * 64, a.vocab, a.w_stride, 64, true)
                     : encode(&t.w_own, DT, a.w, a.cols, a.vocab, a.w_stride, 64);
  constexpr uint64_t es = ra::Elem<WDT>::kSize;
  const bool chunks = (reinterpret_cast<uintptr_t>(a.dweight) | a.dweight_stride * es | a.cols * es) % 16 == 0 && a.dweight_stride < 1ull << 38;
  if (chunks && a.dweight && es == 2 && !a.accumulate && err == cudaSuccess) err = encode(&t.dw_store, DT, a.dweight, a.cols, a.vocab, a.dweight_stride, 32);
  for (uint64_t i = 0; i < 2 && i < a.pieces && err == cudaSuccess; ++i) {
    err = encode(&g[i], DT, scratch + p.g[i], a.piece, a.rows_pad, a.piece, a.rows <= ra::kCeFew ? 64 : 128);
    if (err == cudaSuccess) err = encode(&g_own[i], DT, scratch + p.g[i], a.piece, a.rows_pad, a.piece, 64, true);
    if (err == cudaSuccess) err = encode(&g_store[i], DT, scratch + p.g[i], a.piece, a.rows_pad, a.piece, 32);
  }
  if (err == cudaSuccess) err = rows_and_operands<true>(a, s);
  const auto width = [&](uint64_t piece) { return piece >= a.pieces ? 0 : a.vocab - piece * a.piece < a.piece ? a.vocab - piece * a.piece : a.piece; };
  for (uint64_t i = 0; i <= a.pieces && err == cudaSuccess; ++i) {  // piece i of g, and the gradients of the one before
    t.v_out = i * a.piece, t.w_out = width(i), t.g_out = scratch + p.g[i % 2];
    t.v_sum = i ? (i - 1) * a.piece : 0, t.w_sum = i ? width(i - 1) : 0;
    if (i) t.g = g[(i + 1) % 2], t.g_own = g_own[(i + 1) % 2];
    if (i < a.pieces) t.g_store = g_store[i % 2];
    t.counter = a.counters + i;
    t.early = i == 0 && a.rows <= ra::kCeFew && a.w == a.weight;
    const uint64_t rows = a.rows_pad / 256, across = (a.cols + 255) / 256;
    const uint64_t tiles = rows * ((t.w_out + a.words - 1) / a.words) + (a.dhidden && t.w_sum ? rows * across * a.splits : 0) +
                           (a.dweight ? (t.w_sum + 255) / 256 * across : 0);
    err = chunks || !a.dweight ? launch_tiles<DT, WDT, true, true>(t, tiles, s) : launch_tiles<DT, WDT, true, false>(t, tiles, s);
  }
  if (err == cudaSuccess) {
    const uint64_t units = a.dhidden && a.rows ? a.rows * ((a.cols + 3) / 4) : 1;
    err = launch(ra::ce_finish_kernel<DT, WDT>, dim3(at_most((units + 255) / 256, 152 * 64)), 256, s, a);
  }
  return err;
}

char* first_place(void* workspace) { return reinterpret_cast<char*>(ra::round_up(reinterpret_cast<uintptr_t>(workspace), 256)); }

void place(CeArgs& a, const CePlan& p, void* workspace, bool packed) {
  char* w = first_place(workspace);
  a.rows_pad = p.rows_pad, a.cols_pad = p.cols_pad, a.part_rows = p.part_rows, a.parts = p.parts;
  a.words = p.words, a.slots = p.slots, a.piece = p.piece, a.pieces = p.pieces, a.splits = p.splits;
  a.head = reinterpret_cast<ra::CeHeader*>(w);
  a.counters = reinterpret_cast<uint32_t*>(w + p.counters);
  a.tops = reinterpret_cast<float*>(w + p.tops);
  a.index = reinterpret_cast<int32_t*>(w + p.index);
  a.where = reinterpret_cast<int32_t*>(w + p.where);
  a.target = reinterpret_cast<int32_t*>(w + p.target);
  a.h = w + p.hidden;
  a.w = packed ? w + p.weight : a.weight;
  a.w_stride = packed ? p.cols_pad : a.weight_stride;
  a.lse_kept = reinterpret_cast<float*>(w + p.lse);
  a.dloss_kept = reinterpret_cast<float*>(w + p.dloss);
  a.dh = reinterpret_cast<float*>(w + p.dhidden);
  a.logit = reinterpret_cast<float*>(w + p.logit);
  a.partial = reinterpret_cast<float2*>(w + p.partial);
}

ra_status_t check_type(int dtype) {
  const ra_status_t st = ra::check_float(dtype);
  return st == RA_SUCCESS && dtype == RA_FLOAT32 ? RA_ERR_UNSUPPORTED : st;
}

// RA_SUCCESS if every buffer is sound and no output overlaps another buffer.
template <int IN, int OUT>
ra_status_t check_buffers(Buffer (&in)[IN], Buffer (&out)[OUT], uint64_t width) {
  for (Buffer& b : in)
    if (!ra::sound(b)) return RA_ERR_INVALID_ARG;
  for (Buffer& b : out)
    if (!ra::sound(b)) return RA_ERR_INVALID_ARG;
  for (int o = 0; o < OUT; ++o) {
    for (const Buffer& b : in)
      if (ra::shares(out[o], b, width)) return RA_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (ra::shares(out[o], out[q], width)) return RA_ERR_ALIAS;
  }
  return RA_SUCCESS;
}

ra_status_t call_forward(const void* hidden, size_t hidden_stride, const void* weight,
                         size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                         float* loss, float* lse, size_t rows, size_t cols, size_t vocab,
                         ra_dtype_t dtype, void* workspace, size_t workspace_bytes, const Limits& limits, void* stream) {
  ra_status_t st = check_type(dtype);
  if (st != RA_SUCCESS) return st;
  if ((index_size != 4 && index_size != 8) || cols == 0 || vocab == 0 || !sizes_ok(rows, cols, vocab) ||
      !ra::stride_ok(rows, cols, hidden_stride) || !ra::stride_ok(vocab, cols, weight_stride))
    return RA_ERR_INVALID_ARG;
  if (rows == 0) return RA_SUCCESS;
  const bool packed = !in_place(weight, weight_stride);
  const CePlan p = ra::ce_plan(rows, cols, vocab, packed, false);
  if (workspace_bytes < p.bytes) return RA_ERR_INVALID_ARG;
  Buffer in[3] = {{hidden, ra::extent(rows, cols, hidden_stride, 2), 2, true, {}, hidden_stride * 2},
                  {weight, ra::extent(vocab, cols, weight_stride, 2), 2, true, {}, weight_stride * 2},
                  {targets, rows * index_size, index_size, true, {}}};
  Buffer out[3] = {{loss, rows * 4, 4, true, {}}, {lse, rows * 4, 4, true, {}}, {workspace, p.bytes, 16, true, {}}};
  st = check_buffers(in, out, cols * 2);
  if (st != RA_SUCCESS) return st;
  CeArgs a = {};
  a.hidden = hidden, a.weight = weight, a.hidden_stride = hidden_stride, a.weight_stride = weight_stride;
  a.targets = {targets, (int)index_size}, a.ignore = ignore, a.rows = rows, a.cols = cols, a.vocab = vocab;
  a.loss = loss, a.lse = lse;
  place(a, p, workspace, packed);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return ra::launched(dtype == RA_FLOAT16 ? forward<ra::DT_F16>(a, limits, s) : forward<ra::DT_BF16>(a, limits, s));
}

ra_status_t call_backward(const void* hidden, size_t hidden_stride, const void* weight,
                          size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                          const float* lse, const float* dloss, void* dhidden, size_t dhidden_stride,
                          void* dweight, size_t dweight_stride, int accumulate, size_t rows, size_t cols,
                          size_t vocab, ra_dtype_t dtype, ra_dtype_t dweight_dtype, void* workspace,
                          size_t workspace_bytes, const Limits& limits, void* stream) {
  ra_status_t st = check_type(dtype);
  if (st == RA_SUCCESS) st = ra::check_float(dweight_dtype);
  if (st == RA_SUCCESS && dweight_dtype != dtype && dweight_dtype != RA_FLOAT32) st = RA_ERR_UNSUPPORTED;
  if (st != RA_SUCCESS) return st;
  if ((index_size != 4 && index_size != 8) || cols == 0 || vocab == 0 || !sizes_ok(rows, cols, vocab) ||
      !ra::stride_ok(rows, cols, hidden_stride) || !ra::stride_ok(vocab, cols, weight_stride) ||
      (dhidden && !ra::stride_ok(rows, cols, dhidden_stride)) || (dweight && !ra::stride_ok(vocab, cols, dweight_stride)))
    return RA_ERR_INVALID_ARG;
  if ((!dhidden && !dweight) || (rows == 0 && (!dweight || accumulate))) return RA_SUCCESS;
  const uint64_t ws = ra::float_size(dweight_dtype);
  const bool packed = !in_place(weight, weight_stride);
  const CePlan p = ra::ce_plan(rows, cols, vocab, packed, true);
  if (workspace_bytes < p.bytes) return RA_ERR_INVALID_ARG;
  const auto full = [&](size_t stride) { return rows ? ra::extent(rows, cols, stride, 2) : 0; };
  Buffer in[5] = {{hidden, full(hidden_stride), 2, rows > 0, {}, hidden_stride * 2},
                  {weight, ra::extent(vocab, cols, weight_stride, 2), 2, true, {}, weight_stride * 2},
                  {targets, rows * index_size, index_size, rows > 0, {}},
                  {lse, rows * 4, 4, rows > 0, {}},
                  {dloss, rows * 4, 4, false, {}}};
  Buffer out[3] = {{dhidden, full(dhidden_stride), 2, false, {}, dhidden_stride * 2},
                   {dweight, ra::extent(vocab, cols, dweight_stride, ws), ws, false, {}, dweight_stride * ws},
                   {workspace, p.bytes, 16, true, {}}};
  st = check_buffers(in, out, cols * (ws > 2 ? ws : 2));
  if (st != RA_SUCCESS) return st;
  CeArgs a = {};
  a.hidden = hidden, a.weight = weight, a.hidden_stride = hidden_stride, a.weight_stride = weight_stride;
  a.targets = {targets, (int)index_size}, a.ignore = ignore, a.rows = rows, a.cols = cols, a.vocab = vocab;
  a.lse = const_cast<float*>(lse), a.dloss = dloss;
  a.dhidden = dhidden, a.dweight = dweight, a.dhidden_stride = dhidden_stride, a.dweight_stride = dweight_stride;
  a.accumulate = accumulate != 0;
  place(a, p, workspace, packed);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* const w = first_place(workspace);
  cudaError_t err;
  if (dtype == RA_FLOAT16)
    err = dweight_dtype == RA_FLOAT32 ? backward<ra::DT_F16, ra::DT_F32>(a, p, w, limits, s) : backward<ra::DT_F16, ra::DT_F16>(a, p, w, limits, s);
  else
    err = dweight_dtype == RA_FLOAT32 ? backward<ra::DT_BF16, ra::DT_F32>(a, p, w, limits, s) : backward<ra::DT_BF16, ra::DT_BF16>(a, p, w, limits, s);
  return ra::launched(err);
}

}  // namespace

extern "C" {

size_t ra_cross_entropy_workspace(const void* weight, size_t weight_stride, size_t rows, size_t cols, size_t vocab,
                                  ra_dtype_t dtype, int backward) {
  if (check_type(dtype) != RA_SUCCESS || !sizes_ok(rows, cols, vocab)) return 0;
  return (size_t)ra::ce_plan(rows, cols, vocab, !in_place(weight, weight_stride), backward != 0).bytes;
}

ra_status_t ra_cross_entropy_forward(const void* hidden, size_t hidden_stride, const void* weight,
                                     size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                                     float* loss, float* lse, size_t rows, size_t cols, size_t vocab,
                                     ra_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return call_forward(hidden, hidden_stride, weight, weight_stride, targets, index_size, ignore, loss, lse, rows, cols, vocab,
                      dtype, workspace, workspace_bytes, Limits{}, stream);
}

ra_status_t ra_cross_entropy_backward(const void* hidden, size_t hidden_stride, const void* weight,
                                      size_t weight_stride, const void* targets, size_t index_size, int64_t ignore,
                                      const float* lse, const float* dloss, void* dhidden, size_t dhidden_stride,
                                      void* dweight, size_t dweight_stride, int accumulate, size_t rows, size_t cols,
                                      size_t vocab, ra_dtype_t dtype, ra_dtype_t dweight_dtype, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return call_backward(hidden, hidden_stride, weight, weight_stride, targets, index_size, ignore, lse, dloss, dhidden,
                       dhidden_stride, dweight, dweight_stride, accumulate, rows, cols, vocab, dtype, dweight_dtype,
                       workspace, workspace_bytes, Limits{}, stream);
}

ra_status_t ra_selftest_cross_entropy_timeout(const void* hidden, const void* weight, const int64_t* targets, float* loss,
                                              float* lse, void* dhidden, void* dweight, size_t rows, size_t cols,
                                              size_t vocab, ra_dtype_t dtype, int withhold, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  if (withhold < ra::CE_TILES || withhold > ra::CE_RESULTS) return RA_ERR_INVALID_ARG;
  const Limits limits{1000000, withhold};  // a millisecond
  if (!dhidden && !dweight)
    return call_forward(hidden, cols, weight, cols, targets, 8, -100, loss, lse, rows, cols, vocab, dtype, workspace,
                        workspace_bytes, limits, stream);
  return call_backward(hidden, cols, weight, cols, targets, 8, -100, lse, nullptr, dhidden, cols, dweight, cols, 0, rows, cols,
                       vocab, dtype, dtype, workspace, workspace_bytes, limits, stream);
}

}  // extern "C"
