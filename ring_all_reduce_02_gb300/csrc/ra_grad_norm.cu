// ra_grad_norm: the global 2-norm of many gradient tensors and the factor that
// clips it, in one launch.
//
// One read of every element, two operations each: HBM bounds it. Resident CTAs
// walk over tiles of the tensors; a tile starts on a 32-byte boundary of its
// tensor's memory, so that all but a tensor's first and last vectors are whole.
// Every thread sums squares in fp32 over its share of the tiles, a CTA folds
// its threads' sums in a fixed tree and writes one partial; the CTA that takes
// the last ticket adds the partials in a fixed order in fp64, so the result
// does not depend on the order in which CTAs finish.
#include <math.h>

#include "ra_host.h"
#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"
#include "ra_tensors.cuh"

namespace ra {

constexpr int kNormThreads = 256;
// 456 CTAs (3 on each of 152 SMs) of 256 threads with four 32-byte vectors in flight each. Measured, 354.8 M fp32
// gradients / one layer's 12.6 M bf16 (back to back): 199 us (7.1 TB/s, 105% of the copy bandwidth) / 6.9 us.
// When they were chosen, at 200 / 7.9: two vectors 265 / 8.9, one 445 / 11.7; 1216 CTAs 198 / 11.4 (the last CTA waits
// for more tickets), 304 CTAs 213 / 7.8.
constexpr int kNormUnroll = 4;
constexpr int kNormCtas = 456;
constexpr int kNormSmall = 32;  // tensors in the small and the large table: kernel parameters hold 32,764 bytes
constexpr int kNormLarge = 1024;
// Elements of a tile.
__host__ __device__ constexpr int norm_tile(int es) { return kNormThreads * kNormUnroll * 32 / es; }

struct NormWorkspace {
  uint32_t ticket;  // CTAs that have written their partial; 0 between calls
  uint32_t pad[3];
  float partial[kNormCtas];
};

struct NormScalars {
  int n;
  uint32_t tiles;
  uint32_t written;  // partials that the launches before this one (a longer list of tensors) have written
  int last;          // this launch writes the result
  float prescale, max_norm;
  float* out;
  NormWorkspace* ws;
};
template <int CAP>
struct NormArgs {
  NormScalars s;
  const void* g[CAP];
  uint64_t count[CAP];
  uint32_t tile0[CAP];
};

// The sum over the CTA of one value per thread, in the first warp; the same tree every time.
template <typename T>
__device__ __forceinline__ T cta_sum(T x, T* smem) {
  constexpr int kWarps = kNormThreads / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x / 32] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = smem[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  }
  return x;
}

template <int DT, int CAP>
__global__ void __launch_bounds__(kNormThreads) grad_norm_kernel(const __grid_constant__ NormArgs<CAP> a) {
  pdl_enter();
  const NormScalars& s = a.s;
  __shared__ float sums[kNormThreads / 32];
  __shared__ double last_sums[kNormThreads / 32];
  __shared__ bool finish;
  constexpr int es = Elem<DT>::kSize, V = 32 / es;
  const F2 prescale = twice(s.prescale);
  F2 acc[4] = {0, 0, 0, 0};
  for (uint32_t tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
    const int lo = last_not_above(a.tile0, s.n, tile);
    const char* g = static_cast<const char*>(a.g[lo]);
    const int64_t count = (int64_t)a.count[lo];
    const int64_t first = (int64_t)(tile - a.tile0[lo]) * norm_tile(es) - (int64_t)((reinterpret_cast<uintptr_t>(g) & 31u) / es) +
                          (int64_t)threadIdx.x * V;
    VecT<8> x[kNormUnroll];
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
      const int64_t i = first + u * (kNormThreads * V);
      if (i >= 0 && i + V <= count) {
        x[u] = ld_vec_w<8>(g + i * es);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u].w[k] = 0;
        if (i + V > 0 && i < count) {
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (i + k >= 0 && i + k < count) x[u].w[k * es / 4] |= ld_elem<DT>(g, (uint64_t)(i + k)) << (k * es % 4 * 8);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        F2 f;
        if constexpr (DT == DT_F32) {
          f = pair(__uint_as_float(x[u].w[k]), __uint_as_float(x[u].w[k + 1]));
        } else {
          f = pair(widen16<DT>(x[u].w[k / 2] & 0xffffu), widen16<DT>(x[u].w[k / 2] >> 16));
        }
        f = mul2(f, prescale);
        acc[k / 2 % 4] = fma2(f, f, acc[k / 2 % 4]);
      }
    }
  }
  const float mine = cta_sum(fold2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]))), sums);
  double sum = (double)mine;
  if (gridDim.x > 1 || s.written > 0 || !s.last) {  // one CTA of one launch has it all
    if (threadIdx.x == 0) {
      float* slot = &s.ws->partial[blockIdx.x];
      *slot = blockIdx.x < s.written ? mine + *slot : mine;
      finish = false;
      if (s.last) {
        __threadfence();
        finish = atomicAdd(&s.ws->ticket, 1u) == gridDim.x - 1;
      }
    }
    __syncthreads();
    if (!finish) return;
    __threadfence();
    sum = 0.0;
    for (uint32_t k = threadIdx.x; k < max(s.written, gridDim.x); k += kNormThreads) sum += (double)__ldcg(&s.ws->partial[k]);
    sum = cta_sum(sum, last_sums);
  }
  if (threadIdx.x == 0) {
    const float norm = (float)sqrt(sum);
    const float inf = __int_as_float(0x7f800000);
    s.out[0] = norm;
    s.out[1] = norm < inf ? s.prescale * fminf(__fdiv_rn(s.max_norm, norm + 1e-6f), 1.0f) : __int_as_float(0x7fffffff);
    s.ws->ticket = 0;
  }
}

}  // namespace ra

namespace {

template <int CAP>
ra_status_t launch_all(const void* const* grads, const size_t* counts, int ntensors, int dtype, ra::NormScalars s,
                       cudaStream_t stream) {
  ra::NormArgs<CAP> a;
  const int es = ra::float_size(dtype);
  int i = 0;
  s.written = 0;
  do {
    uint64_t tiles = 0;
    s.n = 0;
    for (; i < ntensors && s.n < CAP; ++i) {
      if (counts[i] == 0) continue;
      const uint64_t past = reinterpret_cast<uintptr_t>(grads[i]) % 32 / es;  // elements past a vector boundary
      const uint64_t more = (counts[i] + past + ra::norm_tile(es) - 1) / ra::norm_tile(es);
      if (tiles + more > 0x7fffffffull) {
        if (s.n == 0) return RA_ERR_UNSUPPORTED;
        break;
      }
      a.g[s.n] = grads[i], a.count[s.n] = counts[i], a.tile0[s.n++] = (uint32_t)tiles;
      tiles += more;
    }
    s.tiles = (uint32_t)tiles;
    s.last = i == ntensors;
    const uint64_t ctas = tiles < (uint64_t)ra::kNormCtas ? (tiles ? tiles : 1) : (uint64_t)ra::kNormCtas;
    a.s = s;
    cudaError_t err;
    if (dtype == RA_FLOAT32)
      err = ra::launch_programmatic(ra::grad_norm_kernel<ra::DT_F32, CAP>, dim3((unsigned)ctas), ra::kNormThreads, 0, stream, a);
    else if (dtype == RA_FLOAT16)
      err = ra::launch_programmatic(ra::grad_norm_kernel<ra::DT_F16, CAP>, dim3((unsigned)ctas), ra::kNormThreads, 0, stream, a);
    else
      err = ra::launch_programmatic(ra::grad_norm_kernel<ra::DT_BF16, CAP>, dim3((unsigned)ctas), ra::kNormThreads, 0, stream, a);
    if (err != cudaSuccess) return ra::cuda_failed(err);
    if (ctas > s.written) s.written = (uint32_t)ctas;
  } while (i < ntensors);
  return RA_SUCCESS;
}

}  // namespace

extern "C" {

size_t ra_grad_norm_workspace(void) { return sizeof(ra::NormWorkspace); }

ra_status_t ra_grad_norm(const void* const* grads, const size_t* counts, int ntensors, ra_dtype_t dtype,
                         double prescale, double max_norm, float* out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const ra_status_t st = ra::check_float(dtype);
  if (st != RA_SUCCESS) return st;
  if (ntensors < 0 || (ntensors > 0 && (grads == nullptr || counts == nullptr))) return RA_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0) || !(fabs(prescale) < INFINITY)) return RA_ERR_INVALID_ARG;
  const uintptr_t w = reinterpret_cast<uintptr_t>(workspace), d = reinterpret_cast<uintptr_t>(out);
  if (w == 0 || w % 16 || workspace_bytes < sizeof(ra::NormWorkspace) || d == 0 || d % 4) return RA_ERR_INVALID_ARG;
  const ra::Range ws{w, w + sizeof(ra::NormWorkspace)}, result{d, d + 8};
  if (ra::overlaps(ws, result)) return RA_ERR_ALIAS;
  const uint64_t es = (uint64_t)ra::float_size(dtype);
  for (int i = 0; i < ntensors; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(grads[i]);
    if ((uint64_t)counts[i] > RA_MAX_COUNT || p == 0 || p % es || p + counts[i] * es < p) return RA_ERR_INVALID_ARG;
    const ra::Range g{p, p + (uintptr_t)(counts[i] * es)};
    if (ra::overlaps(g, ws) || ra::overlaps(g, result)) return RA_ERR_ALIAS;
  }
  ra::NormScalars s{};
  s.prescale = (float)prescale, s.max_norm = (float)max_norm;
  s.out = out, s.ws = static_cast<ra::NormWorkspace*>(workspace);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return ntensors <= ra::kNormSmall ? launch_all<ra::kNormSmall>(grads, counts, ntensors, dtype, s, cs)
                                    : launch_all<ra::kNormLarge>(grads, counts, ntensors, dtype, s, cs);
}

}  // extern "C"
