// ra_embedding_forward / _backward: argument checks, scratch, launch shapes.
#include <float.h>
#include <math.h>

#include "ra_embedding.cuh"
#include "ra_embedding_plan.h"
#include "ra_host.h"

namespace {

using ra::Buffer;

constexpr uint64_t kMostRows = (1ull << 31) - 1024;

bool lines(const void* p, uint64_t stride_bytes) { return (reinterpret_cast<uintptr_t>(p) | stride_bytes) % 16 == 0; }
bool scale_ok(double scale) { return fabs(scale) <= FLT_MAX; }  // what fp32 holds
unsigned ctas(uint64_t units) { return (unsigned)((units + ra::kEmbThreads / 32 - 1) / (ra::kEmbThreads / 32)); }

template <int DT>
cudaError_t forward(ra::EmbForward a, cudaStream_t s) {
  constexpr uint64_t es = ra::Elem<DT>::kSize;
  constexpr int N = 16 / es;
  if (lines(a.table, a.table_stride * es) && lines(a.out, a.out_stride * es) && a.cols % N == 0) {
    constexpr int U = 4;
    a.across = (a.cols + 32 * N * U - 1) / (32 * N * U);
    return ra::launch_programmatic(ra::embedding_forward_kernel<DT, N, U, true>, dim3(ctas(a.rows * a.across)), ra::kEmbThreads, 0, s, a);
  }
  a.across = (a.cols + 255) / 256;
  return ra::launch_programmatic(ra::embedding_forward_kernel<DT, 8, 1, false>, dim3(ctas(a.rows * a.across)), ra::kEmbThreads, 0, s, a);
}

constexpr int kPerLane(int dtype) { return dtype == RA_FLOAT32 ? 4 : 8; }

template <int THREADS, int ITEMS>
cudaError_t sort_one(const ra::EmbBackward& a, unsigned zeros, cudaStream_t s) {
  return ra::launch_programmatic(ra::embedding_sort_kernel<THREADS, ITEMS>, dim3(ra::kEmbCluster + zeros), THREADS, 0, s, a);
}

// Sorts the tokens, and clears the table beside that.
cudaError_t sort(ra::EmbBackward& a, const ra::EmbPlan& p, bool clear, cudaStream_t s) {
  // 32768 x 8192 bf16 into 50257 rows: 270 us a call with 304 CTAs that clear, 243 with 1216. Leaving out the rows that
  // have a token, which the sums write again, cost more in looking for them than their bytes (290).
  const unsigned zeros = clear ? 1216 : 0;
  // no tokens: a table that is cleared, whatever its size, and no launch of no CTAs
  if (a.rows == 0) return ra::launch_programmatic(ra::embedding_count_kernel, dim3(zeros), ra::kEmbThreads, 0, s, a, 0u);
  // As few tokens to a thread as hold them all (12000 / 16384 / 20011 tokens, us a call: 8 to each of 512 threads 25.3 / 30.9 /
  // 32.3; 4, 4 and 6 22.0 / 27.3 / 30.2; twice as many to each of 256 22.3 / 27.5 / 30.7). 4096: 4 to each of 256 15.0, 2 14.0.
  // More threads wait longer at the barriers (8192: 1 to each of 1024 19.4, 4 to each of 256 18.6).
  if (p.one) {
    if (a.rows <= 2048) return sort_one<256, 1>(a, zeros, s);
    if (a.rows <= 4096) return sort_one<256, 2>(a, zeros, s);
    if (a.rows <= 8192) return sort_one<256, 4>(a, zeros, s);
    if (a.rows <= 16384) return sort_one<512, 4>(a, zeros, s);
    return a.rows <= 24576 ? sort_one<512, 6>(a, zeros, s) : sort_one<512, 8>(a, zeros, s);
  }
  cudaError_t err = cudaSuccess;
  for (uint32_t pass = 0; pass < a.passes && err == cudaSuccess; ++pass) {
    err = ra::launch_programmatic(ra::embedding_count_kernel, dim3(a.ctas + (pass == 0 ? zeros : 0)), ra::kEmbThreads, 0, s, a, pass);
    if (err == cudaSuccess) err = ra::launch_programmatic(ra::embedding_scatter_kernel, dim3(a.ctas), ra::kEmbThreads, 0, s, a, pass);
  }
  return err;
}

template <int DT, int WDT, int N, bool VEC, bool ADD>
cudaError_t sums(const ra::EmbBackward& a, int last, cudaStream_t s) {
  const auto kernel = ra::embedding_sum_kernel<DT, WDT, N, VEC, ADD>;
  constexpr size_t smem = ra::kEmbSumSmem<DT, WDT, N, VEC, ADD>;
  if (smem + 1024 > 48 * 1024) {  // beside the static
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  return ra::launch_programmatic(kernel, dim3((unsigned)((uint64_t)a.spans * a.across)), ra::kEmbThreads, smem, s, a, a.keys[last], a.places[last]);
}

template <int DT, int WDT, bool VEC>
cudaError_t backward_lanes(ra::EmbBackward& a, const ra::EmbPlan& p, bool add, cudaStream_t s) {
  constexpr int N = kPerLane(DT);
  if (add && a.rows <= ra::kEmbFew)
    return ra::launch_programmatic(ra::embedding_few_kernel<DT, WDT, N, VEC>, dim3((unsigned)(a.rows * a.across)), ra::kEmbThreads, 0, s, a);
  const cudaError_t err = sort(a, p, !add, s);
  if (err != cudaSuccess || a.rows == 0) return err;
  const int last = p.one ? 0 : (int)(p.passes - 1) % 2;
  return add ? sums<DT, WDT, N, VEC, true>(a, last, s) : sums<DT, WDT, N, VEC, false>(a, last, s);
}

template <int DT, int WDT>
cudaError_t backward(ra::EmbBackward& a, const ra::EmbPlan& p, bool add, cudaStream_t s) {
  const bool vec = lines(a.dy, a.dy_stride * ra::Elem<DT>::kSize) && lines(a.dtable, a.table_stride * ra::Elem<WDT>::kSize) &&
                   a.cols % kPerLane(DT) == 0;
  return vec ? backward_lanes<DT, WDT, true>(a, p, add, s) : backward_lanes<DT, WDT, false>(a, p, add, s);
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
      !scale_ok(scale))
    return RA_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return RA_SUCCESS;
  const uint64_t es = ra::float_size(dtype);
  Buffer t{table, vocab ? ra::extent(vocab, cols, table_stride, es) : 0, es, vocab > 0, {}, table_stride * es};
  Buffer i{tokens, rows * index_size, index_size, true, {}};
  Buffer o{out, ra::extent(rows, cols, out_stride, es), es, true, {}, out_stride * es};
  if (!ra::sound(t) || !ra::sound(i) || !ra::sound(o)) return RA_ERR_INVALID_ARG;
  if (ra::shares(o, t, cols * es) || ra::shares(o, i, cols * es)) return RA_ERR_ALIAS;
  const ra::EmbForward a{table, {tokens, (int)index_size}, out, rows, cols, table_stride, out_stride, 1,
                         (int64_t)vocab, (float)scale, accumulate != 0};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return ra::launched(dtype == RA_FLOAT32   ? forward<ra::DT_F32>(a, s)
                      : dtype == RA_FLOAT16 ? forward<ra::DT_F16>(a, s)
                                            : forward<ra::DT_BF16>(a, s));
}

size_t ra_embedding_workspace(size_t rows, size_t cols, size_t vocab) {
  if (rows > kMostRows || vocab > kMostRows || !ra::shape_ok(rows, cols) || !ra::shape_ok(vocab, cols)) return 0;
  // of the two shapes that a call may take by its type, the larger
  const uint64_t four = ra::emb_plan(rows, cols, vocab, 4).bytes, eight = ra::emb_plan(rows, cols, vocab, 8).bytes;
  return (size_t)(four > eight ? four : eight);
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
      !scale_ok(scale))
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
  const ra::EmbPlan p = ra::emb_plan(rows, cols, vocab, kPerLane(dtype));
  char* const w = static_cast<char*>(workspace);
  const auto at = [&](uint64_t offset) { return reinterpret_cast<uint32_t*>(w + offset); };
  ra::EmbBackward a = {};
  a.dy = dy, a.tokens = {tokens, (int)index_size}, a.dtable = dtable, a.rows = rows, a.cols = cols;
  a.dy_stride = dy_stride, a.table_stride = dtable_stride, a.vocab = (int64_t)vocab, a.padding = padding, a.scale = (float)scale;
  a.bits = p.bits, a.passes = p.passes, a.tiles = (uint32_t)p.tiles, a.ctas = (uint32_t)p.ctas, a.span = (uint32_t)p.span, a.spans = (uint32_t)p.spans;
  a.across = (uint32_t)p.across;
  for (int i = 0; i < 2; ++i) a.keys[i] = at(p.keys[i]), a.places[i] = at(p.places[i]);
  a.counts = at(p.counts), a.tickets = at(p.tickets), a.partial = reinterpret_cast<float*>(w + p.partial);
  a.table_bytes = (int)ws;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool add = accumulate != 0;
  cudaError_t err;
  if (dtype == RA_FLOAT32) err = backward<ra::DT_F32, ra::DT_F32>(a, p, add, s);
  else if (dtype == RA_FLOAT16)
    err = table_dtype == RA_FLOAT32 ? backward<ra::DT_F16, ra::DT_F32>(a, p, add, s) : backward<ra::DT_F16, ra::DT_F16>(a, p, add, s);
  else
    err = table_dtype == RA_FLOAT32 ? backward<ra::DT_BF16, ra::DT_F32>(a, p, add, s) : backward<ra::DT_BF16, ra::DT_BF16>(a, p, add, s);
  return ra::launched(err);
}

}  // extern "C"
