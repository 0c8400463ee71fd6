// Softmax cross entropy from the hidden states h [T, D] and the head's weight w [V, D], in 16 bits.
//
//   forward    logit = h w^T, lse = log sum exp(logit), loss = lse - logit[target]
//   backward   g = dloss (exp(logit - lse) - onehot),  dh = g w,  dw = g^T h
//
// Rows without a loss are left out: a first kernel numbers the others, a second copies their hidden states side by side
// (which also makes them whole 16-byte lines), and every product runs over the rows that count alone. The logits are
// not stored: the forward pass folds every tile of them into a partial maximum and sum per row, which a last kernel
// joins; the backward pass computes them again, a piece of the vocabulary at a time, and stores that piece of g.
#pragma once

#include <cuda_runtime.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"
#include "ra_tokens.cuh"
#include "ra_umma.cuh"

namespace ra {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct CeHeader {
  int32_t rows;  // that count
  int32_t failed; // a wait inside a kernel gave up: every result is NaN
  float scale;   // the largest finite |dloss| (1 if that is 0)
};

// Everything that the kernels need.
struct CeArgs {
  const void *hidden, *weight;  // as given
  const void *h, *w;            // hidden's copy; the weight, or its copy
  uint64_t hidden_stride, weight_stride, w_stride;
  Indices targets;
  int64_t ignore;
  uint64_t rows, cols, vocab, rows_pad, cols_pad, slots, piece;
  CeHeader* head;
  int32_t *index, *where, *target;  // row of a counted row; counted row of a row or -1; its target or -1 (no number of the vocabulary)
  float *lse_kept, *dloss_kept;     // backward: of the counted rows
  float* logit;                     // forward: the target's logit of a counted row
  float2* partial;                  // forward: [rows_pad][slots]
  void* g;                          // backward: [rows_pad][piece]
  float* dh;                        // backward: [rows_pad][cols_pad]
  float *loss, *lse;                // forward: outputs; backward: lse is an input
  const float* dloss;
  void *dhidden, *dweight;
  uint64_t dhidden_stride, dweight_stride;
  int accumulate;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---- rows that count ---------------------------------------------------------------

constexpr int kCeRowsThreads = 1024;

// One CTA: numbers the rows that count in their order.
template <bool BACKWARD>
__global__ void __launch_bounds__(kCeRowsThreads) ce_rows_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  __shared__ int32_t sums[32];
  __shared__ float tops[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int32_t before = 0;
  float top = 0.0f;
  for (uint64_t t0 = 0; t0 < a.rows; t0 += kCeRowsThreads) {
    const uint64_t t = t0 + threadIdx.x;
    const int64_t v = t < a.rows ? load_index(a.targets, t) : a.ignore;
    const bool counts = v != a.ignore;
    const uint32_t votes = __ballot_sync(0xffffffffu, counts);
    if (lane == 0) sums[warp] = __popc(votes);
    __syncthreads();
    int32_t sum = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int32_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    const int32_t all = __shfl_sync(0xffffffffu, sum, 31);
    const int32_t mine = before + (warp ? __shfl_sync(0xffffffffu, sum, warp - 1) : 0) + __popc(votes & ((1u << lane) - 1));
    if (counts) {
      a.index[mine] = (int32_t)t;
      a.target[mine] = v >= 0 && v < (int64_t)a.vocab ? (int32_t)v : -1;
      if constexpr (BACKWARD) {
        const float d = a.dloss ? a.dloss[t] : 1.0f;
        a.lse_kept[mine] = a.lse[t];
        a.dloss_kept[mine] = d;
        if (fabsf(d) < __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(d));
      }
    } else if (!BACKWARD && t < a.rows) {
      a.loss[t] = 0.0f;
      a.lse[t] = 0.0f;
    }
    if (t < a.rows) a.where[t] = counts ? mine : -1;
    before += all;
    __syncthreads();
  }
  if constexpr (BACKWARD) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (threadIdx.x == 0) {
    a.head->rows = before;
    a.head->failed = 0;
    a.head->scale = top > 0.0f ? top : 1.0f;
  }
}

// The counted rows' hidden states side by side, zeros behind them.
__global__ void __launch_bounds__(256) ce_hidden_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const uint64_t rows = (uint64_t)a.head->rows, up = rows ? (rows + 255) / 256 * 256 : 256;
  for (uint64_t i = blockIdx.x; i < up; i += gridDim.x) {
    uint16_t* to = static_cast<uint16_t*>(const_cast<void*>(a.h)) + i * a.cols_pad;
    const uint16_t* from = i < rows ? static_cast<const uint16_t*>(a.hidden) + (uint64_t)a.index[i] * a.hidden_stride : nullptr;
    for (uint64_t c = threadIdx.x; c < a.cols_pad; c += 256) to[c] = from && c < a.cols ? from[c] : (uint16_t)0;
  }
}

// The weight in rows of whole 16-byte lines.
__global__ void __launch_bounds__(256) ce_weight_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  for (uint64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
    uint16_t* to = static_cast<uint16_t*>(const_cast<void*>(a.w)) + v * a.w_stride;
    const uint16_t* from = static_cast<const uint16_t*>(a.weight) + v * a.weight_stride;
    for (uint64_t c = threadIdx.x; c < a.cols_pad; c += 256) to[c] = c < a.cols ? from[c] : (uint16_t)0;
  }
}

// ---- products ------------------------------------------------------------------------
//
// All three products run in one kernel, 256 x 256 elements of the result to a pair of CTAs at a time: a warp brings
// tiles of the operands in by the Tensor Memory Accelerator, a thread issues the products, and 8 warps take the results
// out of tensor memory, which holds two tiles, so that a tile's results are worked on while the next one's products
// run. Every pair takes each so manyth tile.
//   logits  rows x words, summed over the columns     both operands summed-inner
//   dh      rows x columns, summed over the words     g summed-inner, w own-inner
//   dw      words x columns, summed over the rows     g and h own-inner

enum CeKind { CE_LOGITS = 0, CE_G = 1, CE_GRADIENTS = 2 };

constexpr int kCeThreads = 384, kCeOutWarps = 8, kCeStages = 6;
constexpr uint32_t kCeStageBytes = 4 * kBoxBytes;  // 128 x 64 of the one operand, 128 x 64 of the other
constexpr uint32_t kCeSmem = kCeStages * kCeStageBytes + 1024;
constexpr uint32_t kCeGroup = 8;  // tiles of rows that are worked on together, so that the pairs share words and rows

struct CeTiles {
  CUtensorMap h, w, g;
  CeArgs a;
  uint64_t v0, width;  // the words of this launch
};

struct CeTile {
  uint32_t m0, n0;  // first row and column
  uint32_t n;       // columns: 256, or 128 where there are no more
  uint32_t blocks;  // of 64 summed elements
  bool dw;
};

// Tiles of a launch, from the rows that count.
struct CeWork {
  uint32_t rows, row_tiles, col_tiles, words, tiles, dw_tiles, dw_blocks, dh_blocks;
};
template <int KIND>
__device__ __forceinline__ CeWork ce_work(const CeTiles& t) {
  CeWork k;
  k.rows = (uint32_t)t.a.head->rows;
  const uint32_t rows = k.rows ? k.rows : 1;
  k.words = (uint32_t)t.width;
  k.row_tiles = (rows + 255) / 256;
  if constexpr (KIND == CE_GRADIENTS) {
    k.col_tiles = (uint32_t)((t.a.cols + 255) / 256);
    k.dw_blocks = (rows + 63) / 64;
    k.dh_blocks = (k.words + 63) / 64;
    k.dw_tiles = t.a.dweight ? (k.words + 255) / 256 * k.col_tiles : 0;
    k.tiles = k.dw_tiles + (t.a.dhidden ? k.row_tiles * k.col_tiles : 0);
  } else {
    k.col_tiles = (k.words + 255) / 256;
    k.dw_blocks = 0;
    k.dh_blocks = (uint32_t)((t.a.cols + 63) / 64);
    k.dw_tiles = 0;
    k.tiles = k.row_tiles * k.col_tiles;
  }
  return k;
}
template <int KIND>
__device__ __forceinline__ CeTile ce_tile(const CeTiles& t, const CeWork& k, uint32_t i) {
  CeTile o;
  uint32_t m, c, across;
  if constexpr (KIND == CE_GRADIENTS) {
    o.dw = i < k.dw_tiles;
    if (!o.dw) i -= k.dw_tiles;
    m = i / k.col_tiles, c = i % k.col_tiles, across = (uint32_t)t.a.cols;
  } else {
    o.dw = false;
    const uint32_t group = i / (kCeGroup * k.col_tiles), r = i - group * kCeGroup * k.col_tiles;
    const uint32_t left = k.row_tiles - group * kCeGroup, high = left < kCeGroup ? left : kCeGroup;
    m = group * kCeGroup + r % high, c = r / high, across = k.words;
  }
  o.m0 = m * 256, o.n0 = c * 256;
  o.n = across - o.n0 <= 128 ? 128 : 256;
  o.blocks = o.dw ? k.dw_blocks : k.dh_blocks;
  return o;
}

template <int DT>
__device__ __forceinline__ void ce_store(void* p, uint64_t i, float f) {
  if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = f;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)round16<DT>(f);
}
template <int DT>
__device__ __forceinline__ float ce_load(const void* p, uint64_t i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return widen16<DT>(static_cast<const uint16_t*>(p)[i]);
}
// g is held relative to the largest |dloss|, in fp16 times 2^14, where it keeps its digits down to 2^-28 and its
// multiples of 2^-38; both are undone where g has been used.
template <int DT>
__device__ __forceinline__ float ce_unscale(const CeArgs& a) { return a.head->scale * (DT == DT_F16 ? 1.0f / 16384.0f : 1.0f); }
template <int DT>
__device__ __forceinline__ uint32_t ce_pack(float low, float high) {
  uint32_t r;
  if constexpr (DT == DT_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
  return r;
}

// ---- what becomes of a tile's results: a thread has `n` columns (from `col` on) of row `m` in x ----

// The maximum and the sum of exponentials of a row's 128 logits, and the target's logit.
template <int DT>
__device__ __forceinline__ void ce_out_logits(const CeTiles& t, const CeWork& k, uint32_t m, uint32_t col, float (&x)[128]) {
  const float low = __int_as_float(0xff800000);
  if (col + 128 > k.words)
#pragma unroll
    for (int j = 0; j < 128; ++j)
      if (col + j >= k.words) x[j] = low;
  float top = low;
#pragma unroll
  for (int j = 0; j < 128; ++j) top = fmaxf(top, x[j]);
  const float base = top == low ? 0.0f : top;  // a row of -inf alone has the sum 0
  const F2 slope = twice(kLog2e), shift = twice(-base * kLog2e);
  F2 sums[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 128; j += 2) {
    float p, q;
    split(fma2(pair(x[j], x[j + 1]), slope, shift), p, q);
    sums[j / 2 % 4] = add2(sums[j / 2 % 4], pair(exp2_approx(p), exp2_approx(q)));
  }
  if (m >= k.rows) return;
  t.a.partial[(uint64_t)m * t.a.slots + col / 128] = make_float2(top, fold2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]))));
  const uint32_t at = (uint32_t)(t.a.target[m] - (int32_t)col);
  if (at < 128) {
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 128; ++j) y = at == j ? x[j] : y;
    t.a.logit[m] = y;
  }
}

// g = d (exp(logit - lse) - [target]); zero in rows and words behind the last.
template <int DT>
__device__ __forceinline__ void ce_out_g(const CeTiles& t, const CeWork& k, uint32_t m, uint32_t col, float (&x)[128]) {
  const bool counts = m < k.rows;
  const int32_t target = counts ? t.a.target[m] : 0;
  float d = counts ? __fdiv_rn(t.a.dloss_kept[m], t.a.head->scale) * (DT == DT_F16 ? 16384.0f : 1.0f) : 0.0f;
  if (target < 0) d = __int_as_float(0x7fffffff);
  const float shift = counts ? -t.a.lse_kept[m] * kLog2e : 0.0f;
  const F2 slope = twice(kLog2e), both = twice(shift), dd = twice(d);
  const uint32_t at = counts ? (uint32_t)(target - (int32_t)(t.v0 + col)) : 128u;
  float y = 0.0f;
  if (at < 128) {
#pragma unroll
    for (int j = 0; j < 128; ++j) y = at == j ? x[j] : y;
    y = (exp2_approx(__fmaf_rn(y, kLog2e, shift)) - 1.0f) * d;
  }
  uint16_t* to = static_cast<uint16_t*>(t.a.g) + (uint64_t)m * t.a.piece + col;
  const bool ragged = col + 128 > k.words;
#pragma unroll
  for (int j = 0; j < 128; j += 16) {
    VecT<8> v;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float e, f;
      split(fma2(pair(x[j + 2 * q], x[j + 2 * q + 1]), slope, both), e, f);
      split(mul2(pair(exp2_approx(e), exp2_approx(f)), dd), e, f);
      if (ragged) {
        e = col + j + 2 * q < k.words ? e : 0.0f;
        f = col + j + 2 * q + 1 < k.words ? f : 0.0f;
      }
      v.w[q] = ce_pack<DT>(e, f);
    }
    *reinterpret_cast<uint4*>(to + j) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    *reinterpret_cast<uint4*>(to + j + 8) = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
  if (at < 128) to[at] = (uint16_t)round16<DT>(y);
}

template <int DT>
__device__ __forceinline__ void ce_out_dhidden(const CeTiles& t, const CeWork& k, uint32_t m, uint32_t col, float (&x)[128]) {
  if (m >= k.rows) return;
  float* to = t.a.dh + (uint64_t)m * t.a.cols_pad + col;
#pragma unroll
  for (int j = 0; j < 128; j += 4) {
    if (col + j >= t.a.cols_pad) break;
    float4 v = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    if (t.v0) {
      const float4 old = *reinterpret_cast<const float4*>(to + j);
      v = make_float4(v.x + old.x, v.y + old.y, v.z + old.z, v.w + old.w);
    }
    *reinterpret_cast<float4*>(to + j) = v;
  }
}

template <int DT, int WDT>
__device__ __forceinline__ void ce_out_dweight(const CeTiles& t, const CeWork& k, uint32_t m, uint32_t col, float (&x)[128]) {
  if (m >= k.words) return;
  const float scale = ce_unscale<DT>(t.a);
  const uint64_t to = (t.v0 + m) * t.a.dweight_stride + col;
#pragma unroll
  for (int j = 0; j < 128; ++j) {
    if (col + j >= t.a.cols) break;
    float v = x[j] * scale;
    if (t.a.accumulate) v += ce_load<WDT>(t.a.dweight, to + j);
    ce_store<WDT>(t.a.dweight, to + j, v);
  }
}

template <int DT, int WDT, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCeThreads, 1) ce_tiles_kernel(const __grid_constant__ CeTiles t) {
  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t full[kCeStages], empty[kCeStages], ready[2], taken[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int dead;
  uint8_t* const stages = dynamic + (1024u - (smem_u32(dynamic) & 1023u)) % 1024u;  // the swizzle goes by the address
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31, rank = cluster_rank();
  const bool own = KIND == CE_GRADIENTS;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kCeStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ready[i], 1), mbar_init(&taken[i], 2 * kCeOutWarps);
    dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tma_prefetch_map(&t.h);
    tma_prefetch_map(&t.w);
    if (own) tma_prefetch_map(&t.g);
  }
  if (warp == 2) tmem_alloc_pair(&tmem_slot, 512);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_enter();
  const CeWork k = ce_work<KIND>(t);
  const uint32_t first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0 && lane == 0) {
    // the tiles of both operands, each CTA of the pair its half; both count at the even CTA's barrier
    uint32_t s = 0, phase = 0;
    for (uint32_t i = first; i < k.tiles && !dead; i += step) {
      const CeTile o = ce_tile<KIND>(t, k, i);
      const uint32_t half = o.n / 2, boxes = half / 64;
      const int32_t am = (int32_t)(o.m0 + rank * 128), bn = (int32_t)(o.n0 + rank * half);
      for (uint32_t b = 0; b < o.blocks; ++b) {
        if (!mbar_wait_pair(&empty[s], phase ^ 1, &dead)) break;
        uint8_t* const at = stages + s * kCeStageBytes;
        const uint32_t bar = cluster_address(&full[s], 0);
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (2 + boxes) * kBoxBytes);
        const int32_t sum = (int32_t)(b * 64);
        for (uint32_t q = 0; q < 2; ++q) {
          uint8_t* const to = at + q * kBoxBytes;
          if (KIND != CE_GRADIENTS) tma_load_pair(to, &t.h, sum, am + (int32_t)q * 64, bar);
          else if (o.dw) tma_load_pair(to, &t.g, am + (int32_t)q * 64, sum, bar);
          else tma_load_pair(to, &t.g, sum, am + (int32_t)q * 64, bar);
        }
        for (uint32_t q = 0; q < boxes; ++q) {
          uint8_t* const to = at + (2 + q) * kBoxBytes;
          const int32_t col = bn + (int32_t)q * 64;
          if (KIND != CE_GRADIENTS) tma_load_pair(to, &t.w, sum, (int32_t)t.v0 + col, bar);
          else if (o.dw) tma_load_pair(to, &t.h, col, sum, bar);
          else tma_load_pair(to, &t.w, col, (int32_t)t.v0 + sum, bar);
        }
        if (++s == kCeStages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // the products of both CTAs
    uint32_t s = 0, phase = 0, n = 0;
    for (uint32_t i = first; i < k.tiles && !dead; i += step, ++n) {
      const CeTile o = ce_tile<KIND>(t, k, i);
      const uint32_t buffer = n & 1, d = tmem + buffer * 256;
      if (!mbar_wait_pair(&taken[buffer], (n >> 1 & 1) ^ 1, &dead)) break;
      tmem_fence_after();
      const bool a_own = o.dw, b_own = own;
      const uint32_t instruction = umma_instruction(DT == DT_BF16, a_own, b_own, o.n);
      const uint32_t a_step = umma_step(a_own), b_step = umma_step(b_own);
      for (uint32_t b = 0; b < o.blocks; ++b) {
        if (!mbar_wait_pair(&full[s], phase, &dead)) break;
        tmem_fence_after();
        const uint32_t at = smem_u32(stages + s * kCeStageBytes);
        const uint64_t da = umma_descriptor(at, a_own), db = umma_descriptor(at + 2 * kBoxBytes, b_own);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) umma_pair(d, da + q * a_step, db + q * b_step, instruction, b > 0 || q > 0);
        umma_commit_pair(&empty[s]);
        if (++s == kCeStages) s = 0, phase ^= 1;
      }
      umma_commit_pair(&ready[buffer]);
    }
  } else if (warp >= 4) {
    // the results: warp w has lanes 32 (w % 4) on of tensor memory, the first four warps columns 0 to 127
    const uint32_t part = (warp & 3) * 32, col = (warp - 4) / 4 * 128;
    uint32_t n = 0;
    for (uint32_t i = first; i < k.tiles && !dead; i += step, ++n) {
      const CeTile o = ce_tile<KIND>(t, k, i);
      const uint32_t buffer = n & 1;
      if (!mbar_wait_pair(&ready[buffer], n >> 1 & 1, &dead)) break;
      __syncwarp();
      tmem_fence_after();
      float x[128];
      uint32_t* const raw = reinterpret_cast<uint32_t*>(x);
      const uint32_t at = tmem + buffer * 256 + col + (part << 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_load32(at + q * 32, raw + q * 32);
      tmem_wait_loads();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(cluster_address(&taken[buffer], 0));
      const uint32_t m = o.m0 + rank * 128 + part + lane;
      if constexpr (KIND == CE_LOGITS) ce_out_logits<DT>(t, k, m, o.n0 + col, x);
      else if (col < o.n) {
        if constexpr (KIND == CE_G) ce_out_g<DT>(t, k, m, o.n0 + col, x);
        else if (o.dw) ce_out_dweight<DT, WDT>(t, k, m, o.n0 + col, x);
        else ce_out_dhidden<DT>(t, k, m, o.n0 + col, x);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (dead) {  // a wait gave up: the copies and products in flight end first, and the caller sees NaN
    const uint64_t start = global_ns();
    while (global_ns() - start < 10000000ull) {}
    if (threadIdx.x == 0) atomicExch(&t.a.head->failed, 1);
  }
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  if (warp == 2) tmem_free_pair(tmem, 512);
}

// Joins a row's partial sums: a warp per counted row.
__global__ void __launch_bounds__(256) ce_join_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const uint64_t i = (uint64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (i >= (uint64_t)a.head->rows) return;
  const int lane = threadIdx.x & 31;
  const float low = __int_as_float(0xff800000);
  float top = low, sum = 0.0f;
  for (uint64_t s = lane; s < a.slots; s += 32) {
    const float2 p = a.partial[i * a.slots + s];
    const float both = fmaxf(top, p.x), base = both == low ? 0.0f : both;
    sum = sum * exp2_approx((top - base) * kLog2e) + p.y * exp2_approx((p.x - base) * kLog2e);
    top = both;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, top, o), osum = __shfl_xor_sync(0xffffffffu, sum, o);
    const float both = fmaxf(top, other), base = both == low ? 0.0f : both;
    sum = sum * exp2_approx((top - base) * kLog2e) + osum * exp2_approx((other - base) * kLog2e);
    top = both;
  }
  if (lane == 0) {
    const bool there = a.target[i] >= 0 && !a.head->failed;
    const float nan = __int_as_float(0x7fffffff);
    const float lse = there ? top + logf(sum) : nan;
    const uint64_t t = (uint64_t)a.index[i];
    a.lse[t] = lse;
    a.loss[t] = there ? lse - a.logit[i] : nan;
  }
}

// dh into the rows it belongs to, zeros into those that do not count.
template <int DT>
__global__ void __launch_bounds__(256) ce_finish_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const float scale = a.head->failed ? __int_as_float(0x7fffffff) : ce_unscale<DT>(a);
  for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const int32_t i = a.where[t];
    for (uint64_t c = threadIdx.x; c < a.cols; c += 256)
      ce_store<DT>(a.dhidden, t * a.dhidden_stride + c, i < 0 ? 0.0f : a.dh[(uint64_t)i * a.cols_pad + c] * scale);
  }
}

}  // namespace ra
