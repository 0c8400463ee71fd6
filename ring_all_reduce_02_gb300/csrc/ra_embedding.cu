// ra_embedding_forward / _backward: the lookup of a token's row with scaling, and
// the sum of the rows of dy over the places of each token.
#include <math.h>

#include "ra_host.h"
#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_tokens.cuh"

namespace ra {

constexpr int kEmbThreads = 256;

struct EmbForward {
  const void* table;
  Indices tokens;
  void* out;
  uint64_t rows, cols, table_stride, out_stride;
  int64_t vocab;
  float scale;
  int accumulate;
};

template <int DT>
__device__ __forceinline__ float load_float(const void* p, uint64_t i) {
  const uint32_t v = ld_elem<DT>(p, i);
  if constexpr (DT == DT_F32) return __uint_as_float(v);
  else return widen16<DT>(v);
}
template <int DT>
__device__ __forceinline__ void store_float(void* p, uint64_t i, float f) {
  if constexpr (DT == DT_F32) st_elem<DT>(p, i, __float_as_uint(f));
  else st_elem<DT>(p, i, round16<DT>(f));
}

template <int DT>
__global__ void __launch_bounds__(kEmbThreads) embedding_forward_kernel(const __grid_constant__ EmbForward a) {
  pdl_enter();
  const float nan = __int_as_float(0x7fffffff);
  for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const int64_t v = load_index(a.tokens, t);
    const bool there = v >= 0 && v < a.vocab;
    for (uint64_t c = threadIdx.x; c < a.cols; c += kEmbThreads) {
      const uint64_t at = t * a.out_stride + c;
      float x = there ? __fmul_rn(a.scale, load_float<DT>(a.table, (uint64_t)v * a.table_stride + c)) : nan;
      if (a.accumulate) x += load_float<DT>(a.out, at);
      store_float<DT>(a.out, at, x);
    }
  }
}

struct EmbBackward {
  const void* dy;
  Indices tokens;
  void* dtable;
  uint64_t rows, cols, dy_stride, table_stride;
  int64_t vocab, padding;
  float scale;
  int accumulate;
};

// A CTA per row of the table walks over all tokens and adds the rows of dy whose token is its own, in their order.
template <int DT, int WDT>
__global__ void __launch_bounds__(kEmbThreads) embedding_backward_kernel(const __grid_constant__ EmbBackward a) {
  pdl_enter();
  const int64_t v = blockIdx.x;
  for (uint64_t c0 = 0; c0 < a.cols; c0 += kEmbThreads) {
    const uint64_t c = c0 + threadIdx.x;
    float sum = 0.0f;
    bool any = false;
    if (v != a.padding) {
      for (uint64_t t0 = 0; t0 < a.rows; t0 += 32) {
        const uint64_t mine = t0 + (threadIdx.x & 31);
        uint32_t hits = __ballot_sync(0xffffffffu, mine < a.rows && load_index(a.tokens, mine) == v);
        any |= hits != 0;
        for (; hits; hits &= hits - 1)
          if (c < a.cols) sum += load_float<DT>(a.dy, (t0 + __ffs(hits) - 1) * a.dy_stride + c);
      }
    }
    if (c < a.cols && (any || !a.accumulate)) {
      const uint64_t at = (uint64_t)v * a.table_stride + c;
      float x = __fmul_rn(a.scale, sum);
      if (a.accumulate) x += load_float<WDT>(a.dtable, at);
      store_float<WDT>(a.dtable, at, x);
    }
  }
}

}  // namespace ra

namespace {

using ra::Buffer;

constexpr uint64_t kMostRows = (1ull << 31) - 1024;

template <int DT>
cudaError_t forward(const ra::EmbForward& a, cudaStream_t s) {
  const unsigned ctas = (unsigned)(a.rows < 152 * 64 ? a.rows : 152 * 64);
  return ra::launch_programmatic(ra::embedding_forward_kernel<DT>, dim3(ctas), ra::kEmbThreads, 0, s, a);
}
template <int DT, int WDT>
cudaError_t backward(const ra::EmbBackward& a, cudaStream_t s) {
  return ra::launch_programmatic(ra::embedding_backward_kernel<DT, WDT>, dim3((unsigned)a.vocab), ra::kEmbThreads, 0, s, a);
}

}  // namespace

extern "C" {

ra_status_t ra_embedding_forward(const void* table, size_t table_stride, const void* tokens, size_t index_size,
                                 void* out, size_t out_stride, int accumulate, size_t rows, size_t cols, size_t vocab,
                                 double scale, ra_dtype_t dtype, void* stream) {
  const ra_status_t st = ra::check_float(dtype);
  if (st != RA_SUCCESS) return st;
  if ((index_size != 4 && index_size != 8) || rows > kMostRows || vocab > kMostRows || !ra::shape_ok(rows, cols) ||
      !ra::shape_ok(vocab, cols) || !ra::stride_ok(vocab, cols, table_stride) || !ra::stride_ok(rows, cols, out_stride) ||
      !(fabs(scale) < INFINITY))
    return RA_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RA_SUCCESS;
  const uint64_t es = ra::float_size(dtype);
  Buffer t{table, vocab ? ra::extent(vocab, cols, table_stride, es) : 0, es, vocab > 0, {}, table_stride * es};
  Buffer i{tokens, rows * index_size, index_size, true, {}};
  Buffer o{out, ra::extent(rows, cols, out_stride, es), es, true, {}, out_stride * es};
  if (!ra::sound(t) || !ra::sound(i) || !ra::sound(o)) return RA_ERR_INVALID_ARG;
  if (ra::shares(o, t, cols * es) || ra::shares(o, i, cols * es)) return RA_ERR_ALIAS;
  const ra::EmbForward a{table, {tokens, (int)index_size}, out, rows, cols, table_stride, out_stride, (int64_t)vocab,
                         (float)scale, accumulate != 0};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return ra::launched(dtype == RA_FLOAT32   ? forward<ra::DT_F32>(a, s)
                      : dtype == RA_FLOAT16 ? forward<ra::DT_F16>(a, s)
                                            : forward<ra::DT_BF16>(a, s));
}

size_t ra_embedding_workspace(size_t rows, size_t cols, size_t vocab) {
  if (rows > kMostRows || vocab > kMostRows || !ra::shape_ok(rows, cols) || !ra::shape_ok(vocab, cols)) return 0;
  return 16;
}

ra_status_t ra_embedding_backward(const void* dy, size_t dy_stride, const void* tokens, size_t index_size,
                                  int64_t padding, void* dtable, size_t dtable_stride, int accumulate, size_t rows,
                                  size_t cols, size_t vocab, double scale, ra_dtype_t dtype, ra_dtype_t table_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  ra_status_t st = ra::check_float(dtype);
  if (st == RA_SUCCESS) st = ra::check_float(table_dtype);
  if (st == RA_SUCCESS && table_dtype != dtype && table_dtype != RA_FLOAT32) st = RA_ERR_UNSUPPORTED;
  if (st != RA_SUCCESS) return st;
  if ((index_size != 4 && index_size != 8) || rows > kMostRows || vocab > kMostRows || !ra::shape_ok(rows, cols) ||
      !ra::shape_ok(vocab, cols) || !ra::stride_ok(rows, cols, dy_stride) || !ra::stride_ok(vocab, cols, dtable_stride) ||
      !(fabs(scale) < INFINITY))
    return RA_ERR_INVALID_ARG;
  if (vocab == 0 || cols == 0 || (rows == 0 && accumulate)) return RA_SUCCESS;
  const uint64_t es = ra::float_size(dtype), ws = ra::float_size(table_dtype);
  const uint64_t scratch = ra_embedding_workspace(rows, cols, vocab);
  if (workspace_bytes < scratch) return RA_ERR_INVALID_ARG;
  Buffer in[2] = {{dy, rows ? ra::extent(rows, cols, dy_stride, es) : 0, es, rows > 0, {}, dy_stride * es},
                  {tokens, rows * index_size, index_size, rows > 0, {}}};
  Buffer out[2] = {{dtable, ra::extent(vocab, cols, dtable_stride, ws), ws, true, {}, dtable_stride * ws},
                   {workspace, scratch, 16, true, {}}};
  if (!ra::sound(in[0]) || !ra::sound(in[1]) || !ra::sound(out[0]) || !ra::sound(out[1])) return RA_ERR_INVALID_ARG;
  const uint64_t width = cols * (es > ws ? es : ws);
  for (Buffer& o : out)
    if (ra::shares(o, in[0], width) || ra::shares(o, in[1], width)) return RA_ERR_ALIAS;
  if (ra::shares(out[0], out[1], width)) return RA_ERR_ALIAS;
  const ra::EmbBackward a{dy, {tokens, (int)index_size}, dtable, rows, cols, dy_stride, dtable_stride, (int64_t)vocab,
                          padding, (float)scale, accumulate != 0};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == RA_FLOAT32) err = backward<ra::DT_F32, ra::DT_F32>(a, s);
  else if (dtype == RA_FLOAT16)
    err = table_dtype == RA_FLOAT32 ? backward<ra::DT_F16, ra::DT_F32>(a, s) : backward<ra::DT_F16, ra::DT_F16>(a, s);
  else
    err = table_dtype == RA_FLOAT32 ? backward<ra::DT_BF16, ra::DT_F32>(a, s) : backward<ra::DT_BF16, ra::DT_BF16>(a, s);
  return ra::launched(err);
}

}  // extern "C"
