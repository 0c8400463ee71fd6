// Softmax cross entropy from the hidden states h [T, D] and the head's weight w [V, D], in 16 bits.
//
//   forward    logit = h w^T, lse = log sum exp(logit), loss = lse - logit[target]
//   backward   g = dloss (exp(logit - lse) - onehot),  dh = g w,  dw = g^T h
//
// Rows without a loss are left out: a first kernel copies the hidden states of the others side by side (which also
// makes them whole 16-byte lines), and every product runs over the rows that count alone. The logits are not stored:
// the forward pass folds every tile of them into a partial maximum and sum per row, which a last kernel joins; the
// backward pass computes them again, a piece of the vocabulary at a time, and stores that piece of g.
#pragma once

#include <cuda_runtime.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_pairs.cuh"
#include "ra_tokens.cuh"
#include "ra_umma.cuh"

namespace ra {

constexpr float kLog2e = 1.4426950408889634f;

struct CeHeader {
  int32_t rows;    // that count
  int32_t failed;  // not 0: a wait inside a kernel gave up (CeWait, and where), and every result is NaN
  float scale;     // what g is held relative to (from the first launch on)
};

// Everything that the kernels need.
struct CeArgs {
  const void *hidden, *weight;  // as given
  const void *h, *w;            // hidden's copy; the weight, or its copy
  uint64_t hidden_stride, weight_stride, w_stride;
  Indices targets;
  int64_t ignore;
  uint64_t rows, cols, vocab, rows_pad, cols_pad, part_rows, parts, words, slots, piece, pieces, splits;
  CeHeader* head;
  uint32_t* counters;  // of the tiles that a launch's pairs have taken
  float* tops;         // the first kernel's CTAs' largest finite |dloss|
  int32_t *index, *where, *target;  // row of a counted row; counted row of a row or -1; its target or -1 (no word)
  float *lse_kept, *dloss_kept;     // backward: of the counted rows
  float* logit;                     // forward: the target's logit of a counted row
  float2* partial;                  // forward: [rows_pad][slots]
  float* dh;                        // backward: [splits][rows][cols_pad]
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

constexpr int kCeRowsThreads = 256;

// `cols` 16-bit elements from anywhere to a 16-byte boundary by a warp, zeros up to `padded` (whole lines). A line that
// starts off a 16-byte boundary is put together from 5 words, none of which lies wholly outside the row.
__device__ __forceinline__ void ce_copy_row(void* to, const void* from, uint64_t cols, uint64_t padded, int lane) {
  const uint64_t lines = (cols + 7) / 8;
  for (uint64_t i = lines + lane; i < padded / 8; i += 32) static_cast<uint4*>(to)[i] = make_uint4(0, 0, 0, 0);
  const uintptr_t p = reinterpret_cast<uintptr_t>(from);
  if (p % 16 == 0 && cols % 8 == 0) {
    for (uint64_t i = lane; i < lines; i += 32) static_cast<uint4*>(to)[i] = static_cast<const uint4*>(from)[i];
    return;
  }
  const uint32_t* words = reinterpret_cast<const uint32_t*>(p & ~(uintptr_t)3);
  const uint32_t shift = p % 4 * 8;
  const uint64_t reach = (p % 4 + cols * 2 + 3) / 4;  // words that hold elements of the row
  for (uint64_t i = lane; i < lines; i += 32) {
    uint32_t w[5], v[4];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = 4 * i + k < reach ? words[4 * i + k] : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __funnelshift_r(w[k], w[k + 1], shift);
      const uint64_t c = 8 * i + 2 * k;
      if (c + 2 > cols) v[k] &= c < cols ? 0xffffu : 0u;
    }
    static_cast<uint4*>(to)[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Numbers the rows that count in their order. Every CTA has part_rows rows and counts those before them itself: there are 1216
// CTAs at most, so that this grows with the rows alone (a loss of which no row counts, 2^17 x 64 53 us, 2^20 474, 2^22 1930; at
// 1024 columns and 50257 words 2^20 rows' products take over 60 ms).
template <bool BACKWARD>
__global__ void __launch_bounds__(kCeRowsThreads) ce_rows_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  pdl_next();
  constexpr int kWarps = kCeRowsThreads / 32;
  __shared__ int32_t sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint64_t t0 = blockIdx.x * a.part_rows, t1 = t0 + a.part_rows < a.rows ? t0 + a.part_rows : a.rows;
  // the rows on their way while the targets are looked at
  for (uint64_t t = t0 + warp; t < t1; t += kWarps)
    for (uint64_t b = lane * 128; b < a.cols * 2; b += 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.hidden) + t * a.hidden_stride * 2 + b));
  int32_t before = 0;
#pragma unroll 8
  for (uint64_t t = threadIdx.x; t < t0; t += kCeRowsThreads) before += load_index(a.targets, t) != a.ignore;
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) sums[warp] = before;
  __syncthreads();
  before = 0;
  for (int i = 0; i < kWarps; ++i) before += sums[i];
  float top = 0.0f;
  for (uint64_t u = t0; u < t1; u += 32) {  // every warp numbers all rows, and copies each eighth
    const uint64_t t = u + lane;
    const int64_t v = t < t1 ? load_index(a.targets, t) : a.ignore;
    const bool counts = v != a.ignore;
    const uint32_t votes = __ballot_sync(0xffffffffu, counts);
    if (warp == 0) {
      const int32_t mine = before + __popc(votes & ((1u << lane) - 1));
      if (counts) {
        a.index[mine] = (int32_t)t;
        a.target[mine] = v >= 0 && v < (int64_t)a.vocab ? (int32_t)v : -1;
        if constexpr (BACKWARD) {
          const float d = a.dloss ? a.dloss[t] : 1.0f;
          a.lse_kept[mine] = a.lse[t];
          a.dloss_kept[mine] = d;
          if (fabsf(d) < __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(d));
        }
      } else if (!BACKWARD && t < t1) {
        a.loss[t] = 0.0f;
        a.lse[t] = 0.0f;
      }
      if (t < t1) a.where[t] = counts ? mine : -1;
    }
    int32_t to = before;
    for (uint32_t left = votes; left; left &= left - 1, ++to)
      if (to % kWarps == warp)
        ce_copy_row(static_cast<uint16_t*>(const_cast<void*>(a.h)) + (uint64_t)to * a.cols_pad,
                    static_cast<const uint16_t*>(a.hidden) + (u + __ffs(left) - 1) * a.hidden_stride, a.cols, a.cols_pad, lane);
    before += __popc(votes);
  }
  if (BACKWARD && blockIdx.x == gridDim.x - 1) {  // the products sum over whole blocks of 64 rows
    const int32_t up = before ? (before + 63) / 64 * 64 : 64;
    for (int32_t i = before + warp; i < up; i += kWarps)
      for (uint64_t c = lane; c < a.cols_pad / 8; c += 32)
        static_cast<uint4*>(const_cast<void*>(a.h))[(uint64_t)i * (a.cols_pad / 8) + c] = make_uint4(0, 0, 0, 0);
  }
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) {
      a.tops[blockIdx.x] = top;
      if (blockIdx.x == gridDim.x - 1) {
        a.head->rows = before;
        a.head->failed = 0;
      }
    }
  }
  if (blockIdx.x == 0)
    for (uint64_t i = threadIdx.x; i <= a.pieces; i += kCeRowsThreads) a.counters[i] = 0;
}

// The weight in rows of whole 16-byte lines: a warp per row.
__global__ void __launch_bounds__(256) ce_weight_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  pdl_next();
  for (uint64_t v = (uint64_t)blockIdx.x * 8 + threadIdx.x / 32; v < a.vocab; v += (uint64_t)gridDim.x * 8)
    ce_copy_row(static_cast<uint16_t*>(const_cast<void*>(a.w)) + v * a.w_stride,
                static_cast<const uint16_t*>(a.weight) + v * a.weight_stride, a.cols, a.cols_pad, threadIdx.x & 31);
}

// g is held relative to the largest finite |dloss| (1 if that is 0), by a whole warp.
__device__ __forceinline__ float ce_scale(const CeArgs& a) {
  float top = 0.0f;
  for (uint32_t i = threadIdx.x & 31; i < a.parts; i += 32) top = fmaxf(top, a.tops[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top > 0.0f ? top : 1.0f;
}
// fp16 holds g times 2^14, where it keeps its digits down to 2^-28 and its multiples of 2^-38.
template <int DT>
constexpr float kCeShift = DT == DT_F16 ? 16384.0f : 1.0f;
// A sum of such values as the gradient that it is. The power of two goes from the sum, which keeps all its digits, and not
// from the scale: one below 2^-112 would be subnormal after it.
template <int DT>
__device__ __forceinline__ float ce_unscaled(float x, float scale) { return x * (1.0f / kCeShift<DT>) * scale; }

// ---- products ------------------------------------------------------------------------
//
// All three products run in one kernel, 256 x 256 elements of the result to a pair of CTAs at a time: a warp brings
// tiles of the operands in by the Tensor Memory Accelerator, a thread issues the products, and 8 warps take the results
// out of tensor memory, which holds two tiles, so that a tile's results are worked on while the next one's products
// run. A pair's first tile is its own number's; it takes the others from a counter, the longest first.
//   logits  rows x words, summed over the columns     both operands summed-inner
//   dh      rows x columns, summed over the words     g summed-inner, w own-inner
//   dw      words x columns, summed over the rows     g and h own-inner
// A launch of the backward pass has the gradients' tiles of one piece of g and the tiles of the next piece, in
// another buffer: the short ones fill the gaps that the long ones leave at the end.
//
// The tensor pipe bounds a batch: a block of 64 takes 512 cycles of it for 64 KB of operands, and tiles of 256 x 256 over a
// pair halve what each SM reads. 8192 x 1024 x 50257 bf16, logits alone: 403 us for one launch, pipe 97% busy, 2.09
// PFLOP/s; back to back the board's power holds the clock lower, 487 us a call, 1.73 PFLOP/s (a library product of such
// sizes, columns whole 16 bytes, burst / long loop: 1.90 / 1.71). Its backward pass: 1570 us for 2.53 PFLOP, 1.61 PFLOP/s;
// the launches' ends, where pairs run out of tiles, are most of the rest. Few rows are bound by the words' stream: 1 row, 103
// MB in 25 us of a call's 29, with products of which 255 rows of 256 are empty (43% of the pipe); of 61 rows' gradients 79 us,
// the words read twice and dw written once, 309 MB in all.

// A wait that gave up.
enum CeWait { CE_WAIT_EMPTY = 1, CE_WAIT_TILE, CE_WAIT_TAKEN, CE_WAIT_FULL, CE_WAIT_READ, CE_WAIT_READY };
// What the self-test withholds from the other warps: the tiles' numbers, the second operand, the products, or the reading
// of the results.
enum CeWithheld { CE_NOTHING = 0, CE_TILES, CE_OPERAND, CE_PRODUCTS, CE_RESULTS };
enum CeKind { CE_LOGITS = 0, CE_G = 1, CE_DHIDDEN = 2, CE_DWEIGHT = 3, CE_END = 4 };

constexpr int kCeThreads = 384, kCeOutWarps = 8, kCeStages = 6, kCeRing = 4;
constexpr uint32_t kCeStageBytes = 4 * kBoxBytes;  // 128 x 64 of the one operand, 128 x 64 of the other
constexpr uint32_t kCeTurn = 32 * 128;             // a warp's results on their way to other lanes
constexpr uint32_t kCeSmem = kCeStages * kCeStageBytes + kCeOutWarps * kCeTurn + 1024;
constexpr uint32_t kCeLong = 8;   // blocks of a tile that the next one is not taken ahead of
constexpr uint32_t kCeFew = 256;  // rows, at most, that one tile has all of
constexpr uint32_t kCeGroup = 8;  // tiles of rows that are worked on together, so that the pairs share words and rows

struct CeTiles {
  // Boxes of 128 x 64 with rows along the summed dimension (h, w, g: the piece whose gradients are summed; with few rows
  // h's and g's are of 64 rows), and of two groups of 64 with rows along their own (h_own, w_own, g_own). Where w's
  // rows are no whole groups, w_own's boxes are of one.
  CUtensorMap h, w, g, h_own, w_own, g_own;
  CUtensorMap g_store, dw_store;  // boxes of 32 rows of 64 columns
  CeArgs a;
  void* g_out;              // the piece that is computed (forward: none)
  uint64_t v_sum, w_sum;    // first word and words of the one piece (none: 0 words)
  uint64_t v_out, w_out;    // of the other; the forward pass's words
  uint32_t* counter;
  int early;                // the first tiles' words may be asked for before the launch before this one has ended
  int w_groups;             // w_own's boxes are of two groups
  int withheld;             // CeWithheld
  uint64_t wait_ns;         // that a wait takes at most
};

// A tile as it is handed to the warps that work on it.
struct __align__(16) CeTile {
  uint32_t m0, n0;      // first row and column
  uint32_t blocks, b0;  // blocks of 64 summed elements, and the first of them
  uint32_t slot;        // logits: its place in a row of partial sums; dh: the share of the words
  uint16_t kind, n;     // n: columns
  uint32_t pad[2];
};

// Columns of a tile with `left` to go: a half where there are no more.
__device__ __forceinline__ uint32_t ce_width(uint32_t wide, uint32_t left) { return wide == 256 && left <= 128 ? 128 : wide; }

// Tiles of a launch, from the rows that count: dh's and dw's, the longer ones first, then those of logits.
struct CeWork {
  uint32_t rows, row_tiles, across, dh_tiles, dw_tiles, tiles, dh_blocks, dh_share, dw_blocks, out_blocks, out_tiles;
  bool dw_first;
};
__device__ __forceinline__ CeWork ce_work(const CeTiles& t) {
  CeWork k;
  k.rows = (uint32_t)t.a.head->rows;
  const uint32_t rows = k.rows ? k.rows : 1;
  k.row_tiles = (rows + 255) / 256;
  k.across = (uint32_t)((t.a.cols + 255) / 256);
  k.dh_blocks = (uint32_t)((t.w_sum + 63) / 64);
  k.dh_share = (k.dh_blocks + (uint32_t)t.a.splits - 1) / (uint32_t)t.a.splits;
  k.dw_blocks = (rows + 63) / 64;
  k.out_blocks = (uint32_t)((t.a.cols + 63) / 64);
  k.dh_tiles = t.a.dhidden && t.w_sum ? k.row_tiles * k.across * (uint32_t)t.a.splits : 0;
  k.dw_tiles = t.a.dweight && t.w_sum ? (uint32_t)((t.w_sum + 255) / 256) * k.across : 0;
  k.out_tiles = (uint32_t)((t.w_out + t.a.words - 1) / t.a.words);
  k.tiles = t.a.head->failed ? 0 : k.dh_tiles + k.dw_tiles + k.row_tiles * k.out_tiles;
  k.dw_first = k.dw_blocks > k.dh_share;
  return k;
}
template <bool BACKWARD>
__device__ __forceinline__ CeTile ce_tile(const CeTiles& t, const CeWork& k, uint32_t i) {
  CeTile o = {};
  if (i >= k.tiles) {
    o.kind = CE_END;
    return o;
  }
  uint32_t m, c, wide = 256, across = (uint32_t)t.a.cols;
  if (BACKWARD && i < k.dh_tiles + k.dw_tiles) {
    const uint32_t first = k.dw_first ? k.dw_tiles : k.dh_tiles;
    o.kind = (i < first) == k.dw_first ? CE_DWEIGHT : CE_DHIDDEN;
    if (i >= first) i -= first;
    m = i / k.across, c = i % k.across;
    if (o.kind == CE_DWEIGHT) {
      o.blocks = k.dw_blocks;
    } else {
      o.slot = m / k.row_tiles, m %= k.row_tiles;
      o.b0 = o.slot * k.dh_share;
      const uint32_t left = k.dh_blocks > o.b0 ? k.dh_blocks - o.b0 : 0;
      o.blocks = left < k.dh_share ? left : k.dh_share;
    }
  } else {
    o.kind = BACKWARD ? CE_G : CE_LOGITS;
    if constexpr (BACKWARD) i -= k.dh_tiles + k.dw_tiles;
    const uint32_t group = i / (kCeGroup * k.out_tiles), r = i - group * kCeGroup * k.out_tiles;
    const uint32_t left = k.row_tiles - group * kCeGroup, high = left < kCeGroup ? left : kCeGroup;
    m = group * kCeGroup + r % high, c = r / high, across = (uint32_t)t.w_out, wide = (uint32_t)t.a.words;
    o.slot = 2 * c;
    o.blocks = k.out_blocks;
  }
  o.m0 = m * 256, o.n0 = c * wide;
  o.n = (uint16_t)ce_width(wide, across - o.n0);
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
// Results on their way from a lane that holds a row of them to lanes that store 16 bytes each of a few rows: 32 rows of
// 128 bytes in shared memory, 16-byte chunk c of row r at c ^ r % 8. A lane that stored its own row's sectors one by one
// (32 lines an instruction) would keep the SM at 9 bytes a cycle.
__device__ __forceinline__ uint4* ce_chunk(uint8_t* turn, uint32_t row, uint32_t chunk) {
  return reinterpret_cast<uint4*>(turn + row * 128 + (chunk ^ (row & 7)) * 16);
}
// What ce_send sent has left, before the warp puts anything there.
__device__ __forceinline__ void ce_free() {
  if ((threadIdx.x & 31) == 0) tma_stores_read();
  __syncwarp();
}
// The lane's row: 32 words.
__device__ __forceinline__ void ce_put(uint8_t* turn, const uint32_t* w) {
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c) *ce_chunk(turn, threadIdx.x & 31, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
// The 32 rows on their way to box (x, y), while the warp goes on (16 bytes from each lane instead: 17 us more a call of 61 x
// 1024 x 50257 bf16).
__device__ __forceinline__ void ce_send(const CUtensorMap* map, const uint8_t* turn, uint32_t x, uint64_t y) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tma_store(map, turn, (int32_t)x, (int32_t)y);
}
// What of it the lane stores in round i: chunk lane % 8 of row 4 i + lane / 8.
__device__ __forceinline__ uint32_t ce_row_of(uint32_t i) { return 4 * i + (threadIdx.x & 31) / 8; }

// ---- what becomes of a tile's results: a thread has the 128 columns from `col` on of row `m` in x ----

// The maximum and the sum of exponentials of a row's 128 logits, and the target's logit.
__device__ __forceinline__ void ce_out_logits(const CeTiles& t, const CeWork& k, const CeTile& o, uint32_t m, uint32_t col,
                                              float (&x)[128]) {
  const float low = __int_as_float(0xff800000);
  const uint32_t words = o.n0 + o.n < (uint32_t)t.w_out ? o.n0 + o.n : (uint32_t)t.w_out;
  if (col + 128 > words)
#pragma unroll
    for (int j = 0; j < 128; ++j)
      if (col + j >= words) x[j] = low;
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
  t.a.partial[(uint64_t)m * t.a.slots + o.slot + (col > o.n0)] = make_float2(top, fold2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]))));
  const uint32_t at = (uint32_t)(t.a.target[m] - (int32_t)col);
  if (at < 128 && col + at < words) {
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 128; ++j) y = at == j ? x[j] : y;
    t.a.logit[m] = y;
  }
}

// g = d (exp(logit - lse) - [target]), d = dloss / scale; zero in words behind the last and in rows behind the counted
// ones, as far as the products go. The products' operands have 16 bits, so g is rounded to them, once: half a step of the
// operands' type of each g, which is what the gradients differ by from those of an fp32 g (3e-4 of their 2-norm at the
// batch, where bf16's own rounding of them is 1.7e-3). A second product with what the rounding leaves would double the work of dh
// and dw for digits that a 16-bit result cannot hold; with an fp32 dweight it is this rounding that bounds the result. One
// scale for all rows, as dw sums over them: what a row of fp16 has of its range goes by the largest |dloss|.
template <int DT>
__device__ __forceinline__ void ce_out_g(const CeTiles& t, const CeWork& k, const CeTile& o, float scale, uint32_t m, uint32_t col,
                                         float (&x)[64], uint8_t* turn) {
  const uint32_t lane = threadIdx.x & 31, m0 = m - lane, rows = k.dw_blocks * 64;
  if (m0 >= rows) return;
  const bool counts = m < k.rows;
  const int32_t target = counts ? t.a.target[m] : 0;
  float d = counts ? __fdiv_rn(t.a.dloss_kept[m], scale) * kCeShift<DT> : 0.0f;
  if (target < 0) d = __int_as_float(0x7fffffff);
  const float shift = counts ? -t.a.lse_kept[m] * kLog2e : 0.0f;
  const F2 slope = twice(kLog2e), both = twice(shift), dd = twice(d);
  // the last tile goes on to a whole block of 64
  const uint32_t words = (uint32_t)t.w_out, end = o.n0 + o.n < words ? o.n0 + o.n : (words + 63) / 64 * 64;
  if (col >= end) return;
  uint32_t at = counts ? (uint32_t)(target - (int32_t)(t.v_out + col)) : 64u;
  if (at < 64 && col + at >= o.n0 + o.n) at = 64;
  float y = 0.0f;
  if (at < 64) {
#pragma unroll
    for (int j = 0; j < 64; ++j) y = at == j ? x[j] : y;
    y = (exp2_approx(__fmaf_rn(y, kLog2e, shift)) - 1.0f) * d;
  }
  const uint32_t there = !counts || col >= words ? 0 : words - col;
  char* const to = static_cast<char*>(t.g_out) + ((uint64_t)m0 * t.a.piece + col) * 2;
  uint32_t w[32];
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    float e, f;
    split(fma2(pair(x[2 * q], x[2 * q + 1]), slope, both), e, f);
    split(mul2(pair(exp2_approx(e), exp2_approx(f)), dd), e, f);
    w[q] = round16x2<DT>(e, f);
  }
  if (there < 64) {
#pragma unroll
    for (int q = 0; q < 32; ++q) w[q] &= 2 * q + 1 < there ? 0xffffffffu : 2 * q < there ? 0xffffu : 0u;
  }
  ce_free();
  ce_put(turn, w);
  if (at < 64) reinterpret_cast<uint16_t*>(ce_chunk(turn, lane, at / 8))[at % 8] = (uint16_t)round16<DT>(y);
  if (col + 64 <= end) {
    ce_send(&t.g_store, turn, col, m0);
    return;
  }
  __syncwarp();  // the columns behind are another tile's
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) {
    const uint32_t r = ce_row_of(i), c = lane % 8 * 8;
    if (m0 + r < rows && col + c < end) *reinterpret_cast<uint4*>(to + (r * t.a.piece + c) * 2) = *ce_chunk(turn, r, lane % 8);
  }
  __syncwarp();
}

// to[m][col] (+)= x, unscaled as of type DT, for the warp's rows from m0 to `rows` and its columns up to `cols`: rows of
// whole 16-byte chunks. The sums that are added are in flight together. 16-bit results that are not added go through
// `map`, whose row y0 is row 0 here.
template <int DT, int WDT>
__device__ __forceinline__ void ce_out_rows(void* to, uint64_t stride, uint32_t m0, uint32_t rows, uint32_t col, uint32_t cols,
                                            float scale, bool add, float (&x)[64], uint8_t* turn, const CUtensorMap* map, uint64_t y0) {
  constexpr uint32_t es = Elem<WDT>::kSize;
  const uint32_t lane = threadIdx.x & 31;
  if (m0 >= rows || col >= cols) return;
  char* const base = static_cast<char*>(to) + (m0 * stride + col) * es;
  if constexpr (WDT != DT_F32) {
    if (!add) {  // all 64 columns, rounded
      uint32_t w[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) w[q] = round16x2<WDT>(ce_unscaled<DT>(x[2 * q], scale), ce_unscaled<DT>(x[2 * q + 1], scale));
      ce_free();
      ce_put(turn, w);
      ce_send(map, turn, col, y0 + m0);
      return;
    }
  }
  ce_free();
#pragma unroll
  for (uint32_t j = 0; j < 64; j += 32) {
    if (col + j >= cols) break;
    const uint32_t c = j + lane % 8 * 4;
    uint4 old[8];
    if (add) {
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t r = ce_row_of(i);
        old[i] = make_uint4(0, 0, 0, 0);
        if (m0 + r < rows && col + c < cols) {
          const char* at = base + (r * stride + c) * es;
          if constexpr (WDT == DT_F32) {
            old[i] = *reinterpret_cast<const uint4*>(at);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            old[i].x = v.x, old[i].y = v.y;
          }
        }
      }
    }
    uint32_t w[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) w[q] = __float_as_uint(ce_unscaled<DT>(x[j + q], scale));
    ce_put(turn, w);
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = ce_row_of(i);
      const uint4 v = *ce_chunk(turn, r, lane % 8);
      float4 y = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
      if (m0 + r < rows && col + c < cols) {
        char* at = base + (r * stride + c) * es;
        if constexpr (WDT == DT_F32) {
          if (add)
            y = make_float4(y.x + __uint_as_float(old[i].x), y.y + __uint_as_float(old[i].y), y.z + __uint_as_float(old[i].z),
                            y.w + __uint_as_float(old[i].w));
          *reinterpret_cast<float4*>(at) = y;
        } else {
          y = make_float4(y.x + widen16<WDT>(old[i].x & 0xffffu), y.y + widen16<WDT>(old[i].x >> 16),
                          y.z + widen16<WDT>(old[i].y & 0xffffu), y.w + widen16<WDT>(old[i].y >> 16));
          *reinterpret_cast<uint2*>(at) = make_uint2(round16x2<WDT>(y.x, y.y), round16x2<WDT>(y.z, y.w));
        }
      }
    }
    __syncwarp();
  }
}

// dw (+)= scale * x for rows that start anywhere, by a warp and from tensor memory (`at`: its 128 columns; rows m0 on): 32 columns
// at a time are turned in shared memory, so that the warp reads and stores 32 columns of a row together, all 32 rows' in
// flight at once.
template <int DT, int WDT>
__device__ __forceinline__ void ce_out_dweight_turned(const CeTiles& t, float scale, uint32_t m0, uint32_t col, uint32_t at, uint8_t* turn) {
  const uint32_t cols = (uint32_t)t.a.cols, words = (uint32_t)t.w_sum, lane = threadIdx.x & 31;
  const uint32_t high = m0 >= words ? 0 : words - m0 < 32 ? words - m0 : 32;
  ce_free();
#pragma unroll 1
  for (uint32_t j = 0; j < 128 && col + j < cols; j += 32) {
    uint32_t x[32];
    tmem_load32(at + j, x);
    tmem_wait_loads();
    const uint32_t c = col + j + lane, rows = c < cols ? high : 0;
    const uint64_t first = (t.v_sum + m0) * t.a.dweight_stride + c;
    float old[32];
    if (t.a.accumulate) {
#pragma unroll
      for (uint32_t r = 0; r < 32; ++r) old[r] = r < rows ? ce_load<WDT>(t.a.dweight, first + r * t.a.dweight_stride) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < 32; ++q) x[q] = __float_as_uint(ce_unscaled<DT>(__uint_as_float(x[q]), scale));
    ce_put(turn, x);
    __syncwarp();
#pragma unroll
    for (uint32_t r = 0; r < 32; ++r) {
      float v = reinterpret_cast<const float*>(ce_chunk(turn, r, lane / 4))[lane % 4];
      if (t.a.accumulate) v += old[r];
      if (r < rows) ce_store<WDT>(t.a.dweight, first + r * t.a.dweight_stride, v);
    }
    __syncwarp();
  }
}

// A pair's tiles, handed to its warps through a small ring in both CTAs.
struct CeTurns {
  CeTile tile[kCeRing];
  uint64_t full[kCeRing], empty[kCeRing];
};

// CHUNKS: dw's rows are whole 16-byte chunks. The two ways to store it are kernels of their own, so that 16-bit chunks need no
// register more than there are (61 x 1024 x 50257 bf16 85 us a call by one kernel for both, 79 so; 1537 x 768 x 10007 fp16 added
// 74 and 67). The other three still spill: an fp32 dw in chunks 64 bytes a thread, dw off the grid 70 of either type.
template <int DT, int WDT, bool BACKWARD, bool CHUNKS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCeThreads, 1) ce_tiles_kernel(const __grid_constant__ CeTiles t) {
  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t full[kCeStages], empty[kCeStages], ready[2], taken[2];
  __shared__ CeTurns turns;
  __shared__ uint32_t tmem_slot;
  __shared__ int dead;
  uint8_t* const stages = dynamic + (1024u - (smem_u32(dynamic) & 1023u)) % 1024u;  // the swizzle goes by the address
  const uint32_t warp = uniform(threadIdx.x / 32), lane = threadIdx.x & 31, rank = uniform(cluster_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kCeStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ready[i], 1), mbar_init(&taken[i], 2 * kCeOutWarps);
    // a tile's number is read by four loading threads, one that issues products, and both CTAs' warps for the results
    for (int i = 0; i < kCeRing; ++i) mbar_init(&turns.full[i], 1), mbar_init(&turns.empty[i], 5 + 2 * kCeOutWarps);
    dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tma_prefetch_map(&t.h);
    tma_prefetch_map(&t.w);
    if (BACKWARD) tma_prefetch_map(&t.g), tma_prefetch_map(&t.g_own), tma_prefetch_map(&t.h_own), tma_prefetch_map(&t.w_own);
  }
  if (warp == 2) tmem_alloc_pair(&tmem_slot, 512);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = uniform(tmem_slot);
  const bool few = t.a.rows <= kCeFew;
  // With few rows the first tile's words do not depend on how many rows count. Nothing in this call writes them, and
  // what did before it has ended: the launch before this one waited for that before it let this one start.
  uint32_t early = 0;
  if (t.early && warp == 2 && blockIdx.x / 2 * t.a.words < t.w_out) {
    const uint32_t all = (uint32_t)((t.a.cols + 63) / 64);
    const uint32_t n0 = blockIdx.x / 2 * (uint32_t)t.a.words, half = ce_width((uint32_t)t.a.words, (uint32_t)t.w_out - n0) / 2;
    for (; early < all && early < kCeStages; ++early)
      if (elected()) tma_load_pair(stages + early * kCeStageBytes + 2 * kBoxBytes, &t.w, (int32_t)early * 64, (int32_t)(t.v_out + n0 + rank * half),
                    cluster_address(&full[early], 0));
    // the rest of the tile as far as L2 (1 x 1024 x 50257: 30.4 us a call without, 29.1 with; the tiles after it as well:
    // 32.6)
    for (uint32_t b = early; b < all; ++b)
      if (elected()) tma_prefetch(&t.w, (int32_t)b * 64, (int32_t)(t.v_out + n0 + rank * half));
  }
  pdl_enter();
  pdl_next();
  const CeWork k = ce_work(t);

  // Both by a whole warp, with the same answer in all lanes.
  const auto wait = [&](uint64_t* bar, uint32_t parity, int what) { return mbar_wait_warp(bar, parity, &dead, what, t.wait_ns); };
  const auto gave_up = [&] { return uniform((uint32_t)*const_cast<volatile int*>(&dead)) != 0; };
  uint32_t turn = 0;
  // The next tile, by a whole warp. The loading warps and the one of the products ask for it before they work on the one
  // before, so that they do not wait for it. What it says is the same in all lanes, as what these warps count: one lane
  // issues, and finds all it needs in uniform registers (from a branch of one lane each product waits for its operands
  // to be moved there, 75 cycles of the 128 that it takes).
  const auto next = [&] {
    CeTile o;
    const uint32_t slot = turn % kCeRing, round = turn / kCeRing;
    ++turn;
    o.kind = CE_END;
    if (!wait(&turns.full[slot], round & 1, CE_WAIT_TILE)) return o;
    const volatile uint32_t* from = reinterpret_cast<const volatile uint32_t*>(&turns.tile[slot]);
    o.m0 = uniform(from[0]), o.n0 = uniform(from[1]), o.blocks = uniform(from[2]), o.b0 = uniform(from[3]), o.slot = uniform(from[4]);
    const uint32_t both = uniform(from[5]);
    o.kind = (uint16_t)both, o.n = (uint16_t)(both >> 16);
    if (lane == 0) mbar_arrive_at(cluster_address(&turns.empty[slot], 0));
    return o;
  };

  if (warp == 0) {
    // The first operand, 128 rows of each block to each CTA of the pair. What both CTAs bring in counts at the even one's
    // barrier, and its bytes are announced here: those of the first operand that have to come, and all of the second.
    uint32_t s = 0, phase = 0;
    for (CeTile o = next(), after; o.kind != CE_END && !gave_up(); o = after) {
      const bool logits = !BACKWARD || o.kind == CE_G;
      // Boxes of this CTA, and of both. With few rows they are of 64 rows, and those that hold none are left out, but for
      // one of each CTA: one that brings nothing in could not tell a stage that is free from one that is used again.
      uint32_t boxes = 1, bytes = 4 * kBoxBytes;
      if (few && (logits || o.kind == CE_DHIDDEN)) {
        const uint32_t other = k.rows > 192 ? 2 : 1, first = k.rows > 64 ? 2 : 1;
        boxes = rank ? other : first;
        bytes = (first + other) * kBoxBytes;
      }
      bytes += logits ? (uint32_t)t.a.words * 128 : 4 * kBoxBytes;
      const int32_t own = (int32_t)(o.m0 + rank * 128);
      after = next();
      for (uint32_t b = 0; b < o.blocks; ++b) {
        if (!wait(&empty[s], phase ^ 1, CE_WAIT_EMPTY)) break;
        if (elected()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          uint8_t* const at = stages + s * kCeStageBytes;
          const uint32_t bar = cluster_address(&full[s], 0);
          const int32_t sum = (int32_t)((o.b0 + b) * 64);
          if (BACKWARD && o.kind == CE_DWEIGHT) {
            tma_load_pair(at, &t.g_own, 0, sum, own / 64, bar);
          } else {
            const CUtensorMap* const map = BACKWARD && o.kind == CE_DHIDDEN ? &t.g : &t.h;
            tma_load_pair(at, map, sum, own, bar);
            if (boxes > 1) tma_load_pair(at + kBoxBytes, map, sum, own + 64, bar);
          }
        }
        if (++s == kCeStages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 2 && t.withheld != CE_OPERAND) {
    // the second operand
    uint32_t s = 0, phase = 0;
    for (CeTile o = next(), after; o.kind != CE_END && !gave_up(); o = after) {
      const int32_t own = (int32_t)(o.n0 + rank * (o.n / 2));
      after = next();
      for (uint32_t b = 0; b < o.blocks; ++b) {
        if (b >= early) {
          if (!wait(&empty[s], phase ^ 1, CE_WAIT_EMPTY)) break;
          if (elected()) {
            uint8_t* const at = stages + s * kCeStageBytes + 2 * kBoxBytes;
            const uint32_t bar = cluster_address(&full[s], 0);
            const int32_t sum = (int32_t)((o.b0 + b) * 64);
            if (BACKWARD && o.kind == CE_DWEIGHT) {
              tma_load_pair(at, &t.h_own, 0, sum, own / 64, bar);
            } else if (BACKWARD && o.kind == CE_DHIDDEN) {
              if (t.w_groups) {
                tma_load_pair(at, &t.w_own, 0, (int32_t)t.v_sum + sum, own / 64, bar);
              } else {
                tma_load_pair(at, &t.w_own, own, (int32_t)t.v_sum + sum, bar);
                tma_load_pair(at + kBoxBytes, &t.w_own, own + 64, (int32_t)t.v_sum + sum, bar);
              }
            } else {
              tma_load_pair(at, &t.w, sum, (int32_t)t.v_out + own, bar);
            }
          }
        }
        if (++s == kCeStages) s = 0, phase ^= 1;
      }
      early = 0;
    }
  } else if (warp == 1 && rank == 0 && t.withheld != CE_PRODUCTS) {
    // the products of both CTAs
    uint32_t s = 0, phase = 0, n = 0;
    for (CeTile o = next(), after; o.kind != CE_END && !gave_up(); o = after, ++n) {
      after = next();
      const uint32_t buffer = n & 1, d = tmem + buffer * 256;
      if (!wait(&taken[buffer], (n >> 1 & 1) ^ 1, CE_WAIT_TAKEN)) break;
      tmem_fence_after();
      const bool a_own = BACKWARD && o.kind == CE_DWEIGHT, b_own = BACKWARD && o.kind != CE_G;
      const uint32_t instruction = umma_instruction(DT == DT_BF16, a_own, b_own, o.n);
      const uint32_t a_step = umma_step(a_own), b_step = umma_step(b_own);
      for (uint32_t b = 0; b < o.blocks; ++b) {
        if (!wait(&full[s], phase, CE_WAIT_FULL)) break;
        tmem_fence_after();
        if (elected()) {
          const uint32_t at = smem_u32(stages + s * kCeStageBytes);
          const uint64_t da = umma_descriptor(at, a_own), db = umma_descriptor(at + 2 * kBoxBytes, b_own);
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) umma_pair(d, da + q * a_step, db + q * b_step, instruction, b > 0 || q > 0);
          umma_commit_pair(&empty[s]);
        }
        if (++s == kCeStages) s = 0, phase ^= 1;
      }
      if (elected()) umma_commit_pair(&ready[buffer]);
    }
  } else if (warp == 3 && lane == 0 && rank == 0 && t.withheld != CE_TILES) {
    // The tiles. One is taken as late as keeps the others from waiting for it, so that no pair takes tiles that another
    // would get to earlier: after a long one as soon as all warps know the one before, after a short one three ahead.
    const uint32_t pairs = gridDim.x / 2;
    uint32_t ahead = kCeRing;
    for (uint32_t n = 0; !*const_cast<volatile int*>(&dead); ++n) {
      const uint32_t slot = n % kCeRing;
      if (n >= ahead && !mbar_wait_pair(&turns.empty[(n - ahead) % kCeRing], (n - ahead) / kCeRing & 1, &dead, CE_WAIT_READ, t.wait_ns)) break;
      const CeTile o = ce_tile<BACKWARD>(t, k, n == 0 ? blockIdx.x / 2 : pairs + atomicAdd(t.counter, 1u));
      const uint32_t w[8] = {o.m0, o.n0, o.blocks, o.b0, o.slot, (uint32_t)o.kind | (uint32_t)o.n << 16, 0, 0};
      for (uint32_t to = 0; to < 2; ++to) store_pair(cluster_address(&turns.tile[slot], to), w, cluster_address(&turns.full[slot], to));
      if (o.kind == CE_END) break;
      ahead = o.blocks >= kCeLong ? 2 : kCeRing;
    }
  } else if (warp >= 4 && t.withheld != CE_RESULTS) {
    // the results: warp w has lanes 32 (w % 4) on of tensor memory, the first four warps columns 0 to 127
    const uint32_t part = (warp & 3) * 32, col = (warp - 4) / 4 * 128;
    uint8_t* const mine = stages + kCeStages * kCeStageBytes + (warp - 4) * kCeTurn;
    float scale = 1.0f;
    if (BACKWARD) {
      scale = t.w_sum ? t.a.head->scale : ce_scale(t.a);
      if (!t.w_sum && blockIdx.x == 0 && warp == 4 && lane == 0) t.a.head->scale = scale;
    }
    uint32_t n = 0;
    for (CeTile o = next(); o.kind != CE_END && !gave_up(); o = next(), ++n) {
      const uint32_t buffer = n & 1, m = o.m0 + rank * 128 + part + lane;
      if (BACKWARD && o.kind == CE_DWEIGHT && t.a.accumulate && m < t.w_sum && o.n0 + col < t.a.cols) {
        // what the tile is added to, on its way while the products run
        constexpr uint32_t es = Elem<WDT>::kSize;
        const uint32_t left = ((uint32_t)t.a.cols - o.n0 - col < 128 ? (uint32_t)t.a.cols - o.n0 - col : 128) * es;
        const char* at = static_cast<const char*>(t.a.dweight) + ((t.v_sum + m) * t.a.dweight_stride + o.n0 + col) * es;
        for (uint32_t b = 0; b < left; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + b));
      }
      if (!wait(&ready[buffer], n >> 1 & 1, CE_WAIT_READY)) break;
      __syncwarp();
      tmem_fence_after();
      const uint32_t at = tmem + buffer * 256 + col + (part << 16);
      if (BACKWARD && !CHUNKS && o.kind == CE_DWEIGHT) {
        if (col < o.n) ce_out_dweight_turned<DT, WDT>(t, scale, m - lane, o.n0 + col, at, mine);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(cluster_address(&taken[buffer], 0));
        continue;
      }
      const auto release = [&] {
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(cluster_address(&taken[buffer], 0));
      };
      if constexpr (!BACKWARD) {
        float x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_load32(at + q * 32, reinterpret_cast<uint32_t*>(x) + q * 32);
        tmem_wait_loads();
        release();
        ce_out_logits(t, k, o, m, o.n0 + col, x);
      } else {
#pragma unroll 1
        for (uint32_t j = 0; j < 128; j += 64) {
          float x[64];
#pragma unroll
          for (int q = 0; q < 2; ++q) tmem_load32(at + j + q * 32, reinterpret_cast<uint32_t*>(x) + q * 32);
          tmem_wait_loads();
          if (j) release();
          const uint32_t c = o.n0 + col + j;
          if (o.kind == CE_G) {
            ce_out_g<DT>(t, k, o, scale, m, c, x, mine);
          } else if (col + j < o.n) {
            if (o.blocks == 0)  // a share without words
#pragma unroll
              for (int q = 0; q < 64; ++q) x[q] = 0.0f;
            if (o.kind == CE_DHIDDEN)  // a share of dh, on top of what the piece before left
              ce_out_rows<DT_F32, DT_F32>(t.a.dh + o.slot * t.a.rows * t.a.cols_pad, t.a.cols_pad, m - lane, k.rows, c, (uint32_t)t.a.cols_pad, 1.0f,
                                  t.v_sum > 0, x, mine, nullptr, 0);
            else if constexpr (CHUNKS)
              ce_out_rows<DT, WDT>(static_cast<char*>(t.a.dweight) + t.v_sum * t.a.dweight_stride * Elem<WDT>::kSize, t.a.dweight_stride,
                               m - lane, (uint32_t)t.w_sum, c, (uint32_t)t.a.cols, scale, t.a.accumulate, x, mine,
                               &t.dw_store, t.v_sum);
          }
        }
      }
    }
    if (lane == 0) tma_stores_written();
  }
  __syncwarp();
  __syncthreads();
  if (dead) {  // a wait gave up: the copies and products in flight end first, and the caller sees NaN
    const uint64_t start = global_ns();
    while (global_ns() - start < 10000000ull) {}
    if (threadIdx.x == 0) atomicCAS(&t.a.head->failed, 0, dead + 16 * (int)rank + 256 * (int)(blockIdx.x / 2));
    __syncwarp();
  }
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  if (warp == 2) tmem_free_pair(tmem, 512);
}

// A maximum and a sum relative to it, of two.
__device__ __forceinline__ void ce_join(float& top, float& sum, float other, float osum) {
  const float both = fmaxf(top, other), base = both == __int_as_float(0xff800000) ? 0.0f : both;
  sum = sum * exp2_approx((top - base) * kLog2e) + osum * exp2_approx((other - base) * kLog2e);
  top = both;
}

// Joins the rows' partial sums: WARPS warps to a counted row.
template <int WARPS>
__global__ void __launch_bounds__(256) ce_join_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  __shared__ float2 joined[8];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint64_t i = (uint64_t)blockIdx.x * (8 / WARPS) + warp / WARPS;
  const bool there = i < (uint64_t)a.head->rows;
  float top = __int_as_float(0xff800000), sum = 0.0f;
  if (there) {
#pragma unroll 4
    for (uint64_t s = threadIdx.x % (32 * WARPS); s < a.slots; s += 32 * WARPS) {
      const float2 p = a.partial[i * a.slots + s];
      ce_join(top, sum, p.x, p.y);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, top, o), osum = __shfl_xor_sync(0xffffffffu, sum, o);
    ce_join(top, sum, other, osum);
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) joined[warp] = make_float2(top, sum);
    __syncthreads();
    if (warp % WARPS == 0)
      for (int w = 1; w < WARPS; ++w) ce_join(top, sum, joined[warp + w].x, joined[warp + w].y);
  }
  if (there && lane == 0 && warp % WARPS == 0) {
    const bool word = a.target[i] >= 0 && !a.head->failed;
    const float nan = __int_as_float(0x7fffffff);
    const float lse = word ? top + logf(sum) : nan;
    const uint64_t t = (uint64_t)a.index[i];
    a.lse[t] = lse;
    a.loss[t] = word ? lse - a.logit[i] : nan;
  }
}

// dh's shares added up, into the rows they belong to; zeros into those that do not count. A thread has four columns.
// dw is stored by then, but for a launch that failed: then it is NaN too.
template <int DT, int WDT>
__global__ void __launch_bounds__(256) ce_finish_kernel(const __grid_constant__ CeArgs a) {
  pdl_enter();
  const bool failed = a.head->failed != 0;
  if (failed && a.dweight)
    for (uint64_t v = blockIdx.x; v < a.vocab; v += gridDim.x)
      for (uint64_t c = threadIdx.x; c < a.cols; c += 256) ce_store<WDT>(a.dweight, v * a.dweight_stride + c, __int_as_float(0x7fffffff));
  if (a.dhidden == nullptr) return;
  const float scale = failed ? __int_as_float(0x7fffffff) : a.head->scale;
  const uint32_t across = (uint32_t)((a.cols + 3) / 4);
  const uint64_t each = a.rows * a.cols_pad;
  const bool whole = ((reinterpret_cast<uintptr_t>(a.dhidden) | a.dhidden_stride * 2) & 7) == 0;
  for (uint64_t b = (uint64_t)blockIdx.x * 256 + threadIdx.x; b < a.rows * across; b += (uint64_t)gridDim.x * 256) {
    const uint64_t t = b / across, c = b % across * 4;
    const int32_t i = a.where[t];
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= 0) {
      const float* at = a.dh + (uint64_t)i * a.cols_pad + c;
#pragma unroll 8
      for (uint32_t s = 0; s < a.splits; ++s) {
        const float4 v = *reinterpret_cast<const float4*>(at + s * each);
        sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
      }
      sum = make_float4(ce_unscaled<DT>(sum.x, scale), ce_unscaled<DT>(sum.y, scale), ce_unscaled<DT>(sum.z, scale), ce_unscaled<DT>(sum.w, scale));
    }
    uint16_t* const to = static_cast<uint16_t*>(a.dhidden) + t * a.dhidden_stride + c;
    const uint2 w = make_uint2(round16x2<DT>(sum.x, sum.y), round16x2<DT>(sum.z, sum.w));
    if (whole && c + 4 <= a.cols) {
      *reinterpret_cast<uint2*>(to) = w;
    } else {
      to[0] = (uint16_t)w.x;
      if (c + 1 < a.cols) to[1] = (uint16_t)(w.x >> 16);
      if (c + 2 < a.cols) to[2] = (uint16_t)w.y;
      if (c + 3 < a.cols) to[3] = (uint16_t)(w.y >> 16);
    }
  }
}

}  // namespace ra
