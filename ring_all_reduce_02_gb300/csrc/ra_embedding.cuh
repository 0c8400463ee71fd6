// The embedding lookup with scaling, and its gradient: the sum of the rows of dy over the places of each token.
//
// The gradient's sums go by sorted tokens. A stable radix sort gives the places of every token side by side, in their
// order; warps add up spans of sorted places, each a slice of the columns, and write a token's row where its places end
// inside the span. Places that reach over a span's ends leave a partial sum in scratch; the warp that is last to leave
// one of a token's adds them up in the places' order, so that no sum depends on timing.
#pragma once

#include <cuda_runtime.h>

#include "ra_kernels.cuh"
#include "ra_ops.cuh"
#include "ra_tokens.cuh"
#include "ra_umma.cuh"

namespace ra {

template <int DT>
__device__ __forceinline__ float load_float(const void* p, uint64_t i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return widen16<DT>(static_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_float(void* p, uint64_t i, float f) {
  if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = f;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)round16<DT>(f);
}

// A lane's N columns of a row: with VEC side by side in whole 16-byte lines, else every 32nd, one by one. The first is
// column c0 + emb_first, columns from `cols` on are left out.
template <int N, bool VEC>
__device__ __forceinline__ uint32_t emb_first() { return (threadIdx.x & 31) * (VEC ? N : 1); }

// As they lie in memory, to be widened where they are used: rows in flight take half the registers.
template <int DT, int N, bool VEC>
struct EmbRaw {
  uint32_t w[VEC ? N * Elem<DT>::kSize / 4 : N];
  __device__ __forceinline__ void load(const void* row, uint64_t c, uint64_t cols) {
    if constexpr (VEC) {
#pragma unroll
      for (int l = 0; l < N * Elem<DT>::kSize / 16; ++l) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < cols) v = *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + c * Elem<DT>::kSize + l * 16);
        w[4 * l] = v.x, w[4 * l + 1] = v.y, w[4 * l + 2] = v.z, w[4 * l + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        w[k] = 0;
        if (c + 32 * k < cols) {
          if constexpr (DT == DT_F32) w[k] = static_cast<const uint32_t*>(row)[c + 32 * k];
          else w[k] = static_cast<const uint16_t*>(row)[c + 32 * k];
        }
      }
    }
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (DT == DT_F32) return __uint_as_float(w[k]);
    else if constexpr (VEC) return widen16<DT>(k % 2 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
    else return widen16<DT>(w[k]);
  }
};
template <int DT, int N, bool VEC>
__device__ __forceinline__ void emb_store(void* row, uint64_t c, uint64_t cols, const float (&x)[N]) {
  if constexpr (VEC) {
    constexpr int kLines = N * Elem<DT>::kSize / 16, V = 16 / Elem<DT>::kSize;
#pragma unroll
    for (int l = 0; l < kLines; ++l) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (DT == DT_F32) w[k] = __float_as_uint(x[l * V + k]);
        else w[k] = round16x2<DT>(x[l * V + 2 * k], x[l * V + 2 * k + 1]);
      }
      if (c < cols) *reinterpret_cast<uint4*>(static_cast<char*>(row) + c * Elem<DT>::kSize + l * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (c + 32 * k < cols) store_float<DT>(row, c + 32 * k, x[k]);
  }
}

// Which row, and which of the `across` warps side by side on it.
__device__ __forceinline__ void emb_unit(uint64_t unit, uint64_t across, uint64_t& row, uint64_t& slice) {
  if (across == 1) row = unit, slice = 0;
  else if ((unit | across) >> 32 == 0) row = (uint32_t)unit / (uint32_t)across, slice = (uint32_t)unit % (uint32_t)across;
  else row = unit / across, slice = unit % across;
}

// ---- lookup --------------------------------------------------------------------------

constexpr int kEmbThreads = 256;

struct EmbForward {
  const void* table;
  Indices tokens;
  void* out;
  uint64_t rows, cols, table_stride, out_stride, across;
  int64_t vocab;
  float scale;
  int accumulate;
};

// A warp per row and slice of columns; lanes have U times N columns of it, all of them in flight at once. 30011 x 771 fp32
// added to what is there: 38 us a call, 5.7 TB/s, HBM. 8192 x 1024 bf16: 6.6 us, of which the host's part is 6; 8 rows: 6.0.
template <int DT, int N, int U, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embedding_forward_kernel(const __grid_constant__ EmbForward a) {
  pdl_enter();
  constexpr uint64_t es = Elem<DT>::kSize;
  const uint64_t unit = (uint64_t)blockIdx.x * (kEmbThreads / 32) + threadIdx.x / 32;
  uint64_t t, slice;
  emb_unit(unit, a.across, t, slice);
  if (t >= a.rows) return;
  const uint64_t c0 = slice * (32 * N * U) + emb_first<N, VEC>();
  const int64_t v = load_index(a.tokens, t);
  const bool there = v >= 0 && v < a.vocab;
  const char* from = static_cast<const char*>(a.table) + (there ? v : 0) * a.table_stride * es;
  char* to = static_cast<char*>(a.out) + t * a.out_stride * es;
  EmbRaw<DT, N, VEC> raw[U], old[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u].load(from, c0 + u * 32 * N, there ? a.cols : 0);
  if (a.accumulate) {
#pragma unroll
    for (int u = 0; u < U; ++u) old[u].load(to, c0 + u * 32 * N, a.cols);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = there ? __fmul_rn(raw[u].at(k), a.scale) : __int_as_float(0x7fffffff);
      if (a.accumulate) x[k] += old[u].at(k);
    }
    emb_store<DT, N, VEC>(to, c0 + u * 32 * N, a.cols, x);
  }
}

// ---- gradient: what all its kernels get -------------------------------------------------

struct EmbBackward {
  const void* dy;
  Indices tokens;
  void* dtable;
  uint64_t rows, cols, dy_stride, table_stride;
  int64_t vocab, padding;
  float scale;
  uint32_t bits, passes, tiles, ctas, span, spans, across;
  uint32_t *keys[2], *places[2], *counts, *tickets;
  float* partial;  // [spans][2][across][32 * N]: of the places that come from the span before, and that go on into the next
  int table_bytes;  // of dtable's elements
};

// The number that a token is sorted by: `vocab` where it does not count.
__device__ __forceinline__ uint32_t emb_key(const EmbBackward& a, uint64_t t) {
  const int64_t v = load_index(a.tokens, t);
  return v < 0 || v >= a.vocab || v == a.padding ? (uint32_t)a.vocab : (uint32_t)v;
}

// Clears the table: CTA `part` of `parts`, any number of threads.
__device__ __forceinline__ void emb_clear(const EmbBackward& a, uint32_t part, uint32_t parts) {
  const uint64_t es = (uint64_t)a.table_bytes, width = a.cols * es, pitch = a.table_stride * es;
  const uint64_t v0 = (uint64_t)a.vocab * part / parts, v1 = (uint64_t)a.vocab * (part + 1) / parts;
  char* const table = static_cast<char*>(a.dtable);
  if (pitch == width) {  // one run of bytes
    char* const from = table + v0 * pitch;
    char* const to = table + v1 * pitch;
    char* const lo = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(from) + 15) / 16 * 16);
    char* const hi = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(to) / 16 * 16);
    for (char* b = lo + threadIdx.x * 16; b < hi; b += blockDim.x * 16) *reinterpret_cast<uint4*>(b) = make_uint4(0, 0, 0, 0);
    char* const end = lo < to ? lo : to;
    for (char* b = from + threadIdx.x * 2; b < end; b += blockDim.x * 2) *reinterpret_cast<uint16_t*>(b) = 0;
    for (char* b = (hi > end ? hi : end) + threadIdx.x * 2; b < to; b += blockDim.x * 2) *reinterpret_cast<uint16_t*>(b) = 0;
    return;
  }
  const bool lines = ((reinterpret_cast<uintptr_t>(table) | pitch | width) & 15) == 0;
  const uint64_t step = lines ? 16 : es;
  for (uint64_t v = v0 + threadIdx.x / 32; v < v1; v += blockDim.x / 32) {  // a warp per row
    char* const row = table + v * pitch;
    for (uint64_t b = (threadIdx.x & 31) * step; b < width; b += 32 * step) {
      if (lines) *reinterpret_cast<uint4*>(row + b) = make_uint4(0, 0, 0, 0);
      else if (es == 4) *reinterpret_cast<uint32_t*>(row + b) = 0;
      else *reinterpret_cast<uint16_t*>(row + b) = 0;
    }
  }
}

// ---- sort -----------------------------------------------------------------------------
//
// Stable, by digits of `bits` bits from the lowest. A CTA's items stand in the order (warp, round, lane). Within a warp
// an item's rank among those of its digit is what the warp has counted of the digit plus the lanes before it that hold
// it too; the counts of digits, CTAs and warps, summed up in that order, give each warp's first place for each digit.

template <int THREADS>
struct EmbSort {
  static constexpr int kWarps = THREADS / 32;
  uint16_t counts[kWarps][256];  // at most 32768
  uint32_t masks[kWarps][256];   // the lanes that hold a digit
  uint32_t sums[8];
};

// Ranks of a thread's items among the warp's of the same digit (below 1024: two to a word); the warp's counts of digits
// in s.counts. digit(i): of item i. The lanes with an item's digit meet in a word of shared memory: 8192 tokens 18.0 us a
// call against 18.5 with a ballot for each bit of the digit, and with match.any.
template <int THREADS, int ITEMS, class D>
__device__ __forceinline__ void emb_rank(EmbSort<THREADS>& s, D digit, uint32_t (&ranks)[(ITEMS + 1) / 2]) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (uint32_t d = lane; d < 256; d += 32) {
    s.counts[warp][d] = 0;
    s.masks[warp][d] = 0;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t d = digit(i);
    atomicOr(&s.masks[warp][d], 1u << lane);
    __syncwarp();
    const uint32_t same = s.masks[warp][d], old = s.counts[warp][d];
    const uint32_t before = __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (before == 0) {
      s.counts[warp][d] = (uint16_t)(old + __popc(same));
      s.masks[warp][d] = 0;
    }
    __syncwarp();
    if (i % 2 == 0) ranks[i / 2] = old + before;
    else ranks[i / 2] |= (old + before) << 16;
  }
}
template <int N>
__device__ __forceinline__ uint32_t emb_rank_of(const uint32_t (&ranks)[N], int i) { return i % 2 ? ranks[i / 2] >> 16 : ranks[i / 2] & 0xffffu; }

// Thread d < 256: the items of the digits below d in all CTAs, `all` of d. Every thread of the CTA has to come here.
template <int THREADS>
__device__ __forceinline__ uint32_t emb_digits_below(EmbSort<THREADS>& s, uint32_t all) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint32_t sum = all;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t left = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += left;
  }
  if (warp < 8 && lane == 31) s.sums[warp] = sum;
  __syncthreads();
  uint32_t at = sum - all;
  for (uint32_t w = 0; w < warp && w < 8; ++w) at += s.sums[w];
  return at;
}

__device__ __forceinline__ uint32_t peer_load(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_address(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint32_t* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_address(p, rank)), "r"(v) : "memory");
}

constexpr uint32_t kEmbPlaceBits = 15, kEmbCluster = 8;

// The first cluster sorts all tokens, as words of number and place, a share to each CTA; the others clear the table.
// 8192 tokens of 50257 words take two passes and 6 us, which are chains of exchanges through shared memory and between
// the CTAs (one CTA alone 14 us; a launch for each count and scatter 13). Clearing 50257 x 8192 bf16 beside 32768 tokens:
// 112 us, 7.3 TB/s of stores.
template <int THREADS, int ITEMS>
__global__ void __cluster_dims__(kEmbCluster, 1, 1) __launch_bounds__(THREADS) embedding_sort_kernel(const __grid_constant__ EmbBackward a) {
  pdl_enter();
  pdl_next();
  constexpr uint32_t kShare = THREADS * ITEMS;
  __shared__ struct {
    EmbSort<THREADS> sort;
    uint32_t total[256];
    uint32_t words[kShare];
  } s;
  if (blockIdx.x >= kEmbCluster) {
    emb_clear(a, blockIdx.x - kEmbCluster, gridDim.x - kEmbCluster);
    return;
  }
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32, rank = blockIdx.x, first = warp * 32 * ITEMS + lane;
  for (uint32_t i = rank * THREADS + threadIdx.x; i < a.spans * a.across; i += kEmbCluster * THREADS) a.tickets[i] = 0;
  uint32_t word[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t t = rank * kShare + first + i * 32;
    word[i] = t < a.rows ? emb_key(a, t) << kEmbPlaceBits | t : 0xffffffffu;
  }
  for (uint32_t pass = 0; pass < a.passes; ++pass) {
    const uint32_t shift = kEmbPlaceBits + pass * a.bits, mask = (1u << a.bits) - 1;
    uint32_t ranks[(ITEMS + 1) / 2];
    const auto digit = [&](int i) { return word[i] >> shift & mask; };
    emb_rank<THREADS, ITEMS>(s.sort, digit, ranks);
    __syncthreads();
    const uint32_t d = threadIdx.x;
    if (d < 256) {
      uint32_t mine = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) mine += s.sort.counts[w][d];
      s.total[d] = mine;
    }
    cluster_sync();
    uint32_t all = 0, before = 0;
    if (d < 256) {
      uint32_t n[kEmbCluster];
#pragma unroll
      for (uint32_t c = 0; c < kEmbCluster; ++c) n[c] = peer_load(&s.total[d], c);
#pragma unroll
      for (uint32_t c = 0; c < kEmbCluster; ++c) {
        if (c < rank) before += n[c];
        all += n[c];
      }
    }
    uint32_t at = emb_digits_below(s.sort, all) + before;
    if (d < 256) {
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        const uint32_t n = s.sort.counts[w][d];
        s.sort.counts[w][d] = (uint16_t)at;
        at += n;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t to = s.sort.counts[warp][digit(i)] + emb_rank_of(ranks, i);
      peer_store(&s.words[to % kShare], to / kShare, word[i]);
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) word[i] = s.words[first + i * 32];
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t at = rank * kShare + first + i * 32;
    if (at < a.rows) {
      a.keys[0][at] = word[i] >> kEmbPlaceBits;
      a.places[0][at] = word[i] & ((1u << kEmbPlaceBits) - 1);
    }
  }
}

// More tokens than that: a pass is a count of every CTA's digits, and a CTA's items to their places. Pass 0 reads the
// tokens themselves. A CTA finds its first places from the counts of all, 1 KB of each, so that there are 304 of them at most,
// as many as the device holds, which take tiles in a row (into 50257 x 8 fp32, ms a call: a CTA to each tile 0.62 for 2^22 tokens,
// 37.9 for 2^26; 1216 CTAs 0.67 and 8.5, 608 0.53 for 2^22, 304 0.51 and 9.1).
constexpr int kEmbTileItems = 16;
static_assert(kEmbThreads * kEmbTileItems == 4096, "a tile of the plan");

__device__ __forceinline__ void emb_item(const EmbBackward& a, uint32_t pass, uint64_t t, uint32_t& key, uint32_t& place) {
  key = 0xffffffffu, place = 0;
  if (t >= a.rows) return;
  key = pass ? a.keys[(pass - 1) % 2][t] : emb_key(a, t);
  place = pass ? a.places[(pass - 1) % 2][t] : (uint32_t)t;
}

__global__ void __launch_bounds__(kEmbThreads) embedding_count_kernel(const __grid_constant__ EmbBackward a, uint32_t pass) {
  pdl_enter();
  pdl_next();
  __shared__ uint32_t seen[256];  // of each digit
  if (blockIdx.x >= a.ctas) {
    emb_clear(a, blockIdx.x - a.ctas, gridDim.x - a.ctas);
    return;
  }
  if (pass == 0)
    for (uint64_t i = (uint64_t)blockIdx.x * kEmbThreads + threadIdx.x; i < (uint64_t)a.spans * a.across; i += (uint64_t)a.ctas * kEmbThreads)
      a.tickets[i] = 0;
  seen[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 1
  for (uint32_t tile = 0; tile < a.tiles; ++tile) {
    const uint64_t first = ((uint64_t)blockIdx.x * a.tiles + tile) * 4096 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kEmbTileItems; ++i) {
      uint32_t key, place;
      emb_item(a, pass, first + i * kEmbThreads, key, place);
      if (first + i * kEmbThreads < a.rows) atomicAdd(&seen[key >> pass * a.bits & ((1u << a.bits) - 1)], 1u);
    }
  }
  __syncthreads();
  a.counts[(uint64_t)blockIdx.x * 256 + threadIdx.x] = seen[threadIdx.x];
}

__global__ void __launch_bounds__(kEmbThreads) embedding_scatter_kernel(const __grid_constant__ EmbBackward a, uint32_t pass) {
  pdl_enter();
  pdl_next();
  __shared__ EmbSort<kEmbThreads> s;
  __shared__ uint32_t base[256];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  // this CTA's first place for the thread's digit: items of smaller digits, and of this one in CTAs before
  uint32_t all = 0, before = 0;
#pragma unroll 8
  for (uint32_t c = 0; c < a.ctas; ++c) {
    const uint32_t n = a.counts[(uint64_t)c * 256 + threadIdx.x];
    if (c < blockIdx.x) before += n;
    all += n;
  }
  const uint32_t at = emb_digits_below(s, all) + before;
  base[threadIdx.x] = at;
#pragma unroll 1
  for (uint32_t tile = 0; tile < a.tiles; ++tile) {
    const uint64_t first = ((uint64_t)blockIdx.x * a.tiles + tile) * 4096 + warp * 32 * kEmbTileItems + lane;
    uint32_t key[kEmbTileItems], place[kEmbTileItems], ranks[kEmbTileItems / 2];
#pragma unroll
    for (int i = 0; i < kEmbTileItems; ++i) emb_item(a, pass, first + i * 32, key[i], place[i]);
    const auto digit = [&](int i) { return key[i] >> pass * a.bits & ((1u << a.bits) - 1); };
    emb_rank<kEmbThreads, kEmbTileItems>(s, digit, ranks);
    __syncthreads();
    // items of the digit in the warps before this one
    uint32_t run = 0;
    for (int w = 0; w < kEmbThreads / 32; ++w) {
      const uint32_t n = s.counts[w][threadIdx.x];
      s.counts[w][threadIdx.x] = (uint16_t)run;
      run += n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEmbTileItems; ++i)
      if (first + i * 32 < a.rows) {
        const uint32_t to = base[digit(i)] + s.counts[warp][digit(i)] + emb_rank_of(ranks, i);
        a.keys[pass % 2][to] = key[i];
        a.places[pass % 2][to] = place[i];
      }
    if (tile + 1 < a.tiles) {  // the next tile's come behind these
      __syncthreads();
      base[threadIdx.x] += run;
    }
  }
}

// ---- sums -----------------------------------------------------------------------------

// A warp's slice of a row (32 N columns from c0 on) on its way through shared memory, which holds as many rows in flight
// as the memory's latency asks for without a register for them. With VEC a lane copies and reads its own 16-byte lines;
// else lanes copy every 32nd word that holds some of the slice, and read every 32nd element.
template <int DT, int N, bool VEC>
struct EmbSlice {
  static constexpr uint32_t es = Elem<DT>::kSize, kBytes = 32 * N * es + (VEC ? 0 : 16);
  static __device__ __forceinline__ void copy(uint8_t* slot, const void* row, uint64_t c0, uint64_t cols) {
    const uint32_t lane = threadIdx.x & 31, to = (uint32_t)__cvta_generic_to_shared(slot);
    if constexpr (VEC) {
#pragma unroll
      for (uint32_t l = 0; l < N * es / 16; ++l) {
        const uint64_t c = c0 + lane * N;
        if (c < cols)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + lane * N * es + l * 16),
                       "l"(static_cast<const char*>(row) + c * es + l * 16)
                       : "memory");
      }
    } else {
      const uintptr_t first = reinterpret_cast<uintptr_t>(row) + c0 * es, word = first & ~(uintptr_t)3;
      const uint64_t left = cols - c0 < 32 * N ? cols - c0 : 32 * N;
      const uint32_t words = (uint32_t)((first - word + left * es + 3) / 4);
#pragma unroll
      for (uint32_t j = 0; j <= N * es / 4; ++j)
        if (lane + 32 * j < words)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + (lane + 32 * j) * 4), "l"(word + (lane + 32 * j) * 4) : "memory");
    }
  }
  // The lane's columns; those from `cols` on hold anything.
  static __device__ __forceinline__ void read(const uint8_t* slot, const void* row, uint64_t c0, float (&x)[N]) {
    const uint32_t lane = threadIdx.x & 31;
    if constexpr (VEC) {
#pragma unroll
      for (uint32_t l = 0; l < N * es / 16; ++l) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + lane * N * es + l * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (uint32_t k = 0; k < 16 / es; ++k) {
          if constexpr (DT == DT_F32) x[l * 4 + k] = __uint_as_float(w[k]);
          else x[l * 8 + k] = widen16<DT>(k % 2 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
        }
      }
    } else {
      const uint32_t phase = (uint32_t)((reinterpret_cast<uintptr_t>(row) + c0 * es) & 3);
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = load_float<DT>(slot + phase, lane + 32 * k);
    }
  }
};

// dtable's row of a token: scale * sum, with ADD on top of what it holds (`old`).
template <int WDT, int N, bool VEC, bool ADD>
__device__ __forceinline__ void emb_finish(const EmbBackward& a, char* row, uint64_t c, const float (&sum)[N], const float (&old)[N]) {
  float x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = __fmul_rn(sum[k], a.scale);
    if (ADD) x[k] += old[k];
  }
  emb_store<WDT, N, VEC>(row, c, a.cols, x);
}

// How far a condition holds from the warp's n = 0, where it does: the least n > 0 where it no longer holds. It does not come
// back behind that. 32 numbers at a time, side by side, and where all 32 hold in strides 32 times as long, which come down
// again: a token that has all of 2^23 places took 21.7 ms a call by steps of 32 alone (2^20: 1.1), and 7.7 with this (0.75).
template <class C>
__device__ __forceinline__ uint32_t emb_reach(C holds) {
  uint32_t at = 0, stride = 1;
  while (true) {
    const uint32_t run = __ffs(~__ballot_sync(0xffffffffu, holds((uint64_t)at + (uint64_t)((threadIdx.x & 31) + 1) * stride)));
    if (run == 0) {  // all 32
      at += 32 * stride, stride *= 32;
    } else {
      at += (run - 1) * stride;
      if (stride == 1) return at + 1;
      stride /= 32;
    }
  }
}
// The first span that holds places of the token whose places reach from before into `span`, and the last one that holds
// some of the token whose places go on behind `span`.
__device__ __forceinline__ uint32_t emb_first_span(const EmbBackward& a, const uint32_t* keys, uint32_t span, uint32_t key) {
  return span - emb_reach([&](uint64_t n) { return n < span && keys[(span - n) * a.span - 1] == key; });
}
__device__ __forceinline__ uint32_t emb_last_span(const EmbBackward& a, const uint32_t* keys, uint32_t span, uint32_t key) {
  return span + emb_reach([&](uint64_t n) { return (span + n + 1) * a.span < a.rows && keys[(span + n + 1) * a.span] == key; });
}

// A token's places reach over the ends of spans `first` to `last`: adds up what they left, if this warp is the last of
// them to have left something.
template <int WDT, int N, bool VEC, bool ADD>
__device__ __noinline__ void emb_join(const EmbBackward& a, uint32_t first, uint32_t last, uint32_t across, uint32_t key) {
  const uint32_t lane = threadIdx.x & 31;
  __threadfence();
  __syncwarp();
  uint32_t ticket = 0;
  if (lane == 0) ticket = atomicAdd(&a.tickets[(uint64_t)first * a.across + across], 1u);
  if (__shfl_sync(0xffffffffu, ticket, 0) != last - first) return;
  __threadfence();
  const uint64_t c = (uint64_t)across * 32 * N + emb_first<N, VEC>();
  char* const row = static_cast<char*>(a.dtable) + (uint64_t)key * a.table_stride * Elem<WDT>::kSize;
  float sum[N], old[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = old[k] = 0.0f;
  if (ADD) {
    EmbRaw<WDT, N, VEC> raw;
    raw.load(row, c, a.cols);
#pragma unroll
    for (int k = 0; k < N; ++k) old[k] = raw.at(k);
  }
  const uint64_t slot = (uint64_t)a.across * 32 * N;  // floats of a partial sum
  const float4* at = reinterpret_cast<const float4*>(a.partial + ((uint64_t)first * 2 + 1) * slot + (uint64_t)across * 32 * N + lane * N);
  // the first span's last places, then each one's first, 8 at a time
  for (uint32_t f = first; f <= last; f += 8) {
    float4 v[8][N / 4];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint64_t on = (f + i <= last ? f + i : last) - first;
#pragma unroll
      for (int q = 0; q < N / 4; ++q) v[i][q] = __ldcg(at + (on ? 2 * on - 1 : 0) * (slot / 4) + q);
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < N / 4; ++q)
        if (f + i <= last) sum[4 * q] += v[i][q].x, sum[4 * q + 1] += v[i][q].y, sum[4 * q + 2] += v[i][q].z, sum[4 * q + 3] += v[i][q].w;
  }
  emb_finish<WDT, N, VEC, ADD>(a, row, c, sum, old);
}

// A few rows added to the table, in one launch without a sort: a CTA per row and slice of the columns. The first row of
// its token has the sum of all of them, a share to each warp; the others leave. Adding the shares up goes by the warps'
// order. 61 x 1024 bf16: 7.0 us a call, the host's 6 among them (11 by sort and sums).
constexpr uint32_t kEmbFew = 256;
template <int DT, int WDT, int N, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) embedding_few_kernel(const __grid_constant__ EmbBackward a) {
  pdl_enter();
  constexpr uint32_t kWarps = kEmbThreads / 32;
  static_assert(kEmbThreads == kEmbFew, "a token to each thread");
  __shared__ uint32_t counts[kWarps], list[kEmbFew];
  __shared__ float sums[kWarps][N][32];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32, i = threadIdx.x;
  uint64_t t, slice;
  emb_unit(blockIdx.x, a.across, t, slice);
  const uint32_t none = (uint32_t)a.vocab, own = emb_key(a, t), key = i < a.rows ? emb_key(a, i) : none;
  if (own == none || __syncthreads_or(i < t && key == own)) return;
  const uint32_t votes = __ballot_sync(0xffffffffu, key == own);
  if (lane == 0) counts[warp] = __popc(votes);
  __syncthreads();
  uint32_t at = __popc(votes & ((1u << lane) - 1)), n = 0;
  for (uint32_t w = 0; w < kWarps; ++w) {
    if (w < warp) at += counts[w];
    n += counts[w];
  }
  if (key == own) list[at] = i;
  __syncthreads();
  if (warp >= n) return;  // no barrier of the whole CTA below: the warps that stay are counted
  const uint64_t c = slice * 32 * N + emb_first<N, VEC>();
  char* const row = static_cast<char*>(a.dtable) + (uint64_t)own * a.table_stride * Elem<WDT>::kSize;
  EmbRaw<WDT, N, VEC> old;
  if (warp == 0) old.load(row, c, a.cols);
  float sum[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = 0.0f;
#pragma unroll 4
  for (uint32_t j = warp; j < n; j += kWarps) {
    EmbRaw<DT, N, VEC> x;
    x.load(static_cast<const char*>(a.dy) + (uint64_t)list[j] * a.dy_stride * Elem<DT>::kSize, c, a.cols);
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] += x.at(k);
  }
  const uint32_t warps = n < kWarps ? n : kWarps;
  if (warp > 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) sums[warp][k][lane] = sum[k];
  }
  if (warps > 1) asm volatile("bar.sync 1, %0;" ::"r"(warps * 32) : "memory");
  if (warp > 0) return;
  for (uint32_t w = 1; w < warps; ++w) {
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] += sums[w][k][lane];
  }
  float before[N];
#pragma unroll
  for (int k = 0; k < N; ++k) before[k] = old.at(k);
  emb_finish<WDT, N, VEC, true>(a, row, c, sum, before);
}

// Rows that a warp has in flight, as many as let an SM hold 4 CTAs, which is also what their registers are limited for; and a
// partial sum of each warp beside them. 16-bit rows added to an fp32 table, whose slots are half as large again: 8192 x 1024
// bf16 21.5 us a call with 3 rows and 4 CTAs, 23.9 with 5 and 3; 20011 x 515 fp16 33.1 and 33.9; 32768 x 8192 bf16 239 and 241.
template <int DT, int WDT, bool ADD>
constexpr uint32_t kEmbFlight = !ADD ? 8 : DT == WDT ? 5 : 3;
template <int DT, int WDT, int N, bool VEC, bool ADD>
constexpr uint32_t kEmbSumSmem =
    kEmbThreads / 32 * (32 * N * 4 + kEmbFlight<DT, WDT, ADD> * (EmbSlice<DT, N, VEC>::kBytes + (ADD ? EmbSlice<WDT, N, VEC>::kBytes : 0)));

// A CTA per span of sorted places and slice of the columns, a share of the span to each warp. A warp adds its places'
// rows up in their order, and writes a token's row where its places end; with ADD dtable's row comes along with the
// token's last place. Places that reach over the end of a warp's share are joined by the warp in whose share they start,
// and those that reach over the span's ends by the last CTA that has some of them. Spans of sorted places, not a CTA per
// token: text has tokens that come up in a tenth of all places, which would be one CTA's work (8192 x 1024 bf16 14106 us a
// call by the thread that owns a token's column, 18 by spans). 32768 x 8192 bf16: 121 us, 661 MB at 5.5 TB/s, HBM; 8192 x
// 1024 added: 10 us for 50 MB, a chain of keys, rows and two joins with 30% of the warps an SM holds.
template <int DT, int WDT, int N, bool VEC, bool ADD>
__global__ void __launch_bounds__(kEmbThreads, 4) embedding_sum_kernel(const __grid_constant__ EmbBackward a, const uint32_t* keys, const uint32_t* places) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t flight[];
  using From = EmbSlice<DT, N, VEC>;
  using To = EmbSlice<WDT, N, VEC>;
  constexpr uint32_t kWarps = kEmbThreads / 32, kFlight = kEmbFlight<DT, WDT, ADD>, kSlot = From::kBytes + (ADD ? To::kBytes : 0);
  // 228 KB of an SM, of which each CTA takes 1 KB and its variables of a known size
  static_assert(4 * (kEmbSumSmem<DT, WDT, N, VEC, ADD> + 1024 + 128) <= 228 * 1024, "4 CTAs to an SM");
  static_assert(kFlight * kSlot >= 32 * N * 4, "the rows' place takes a partial sum when they are through");
  enum { HEAD = 1, HEAD_ENDS = 2, TAIL = 4 };  // places that come from the share before, and end here; that go on
  __shared__ uint32_t left[kWarps], keys_left[kWarps], first_span, last_span;
  uint64_t row, slice;
  emb_unit(blockIdx.x, a.across, row, slice);
  const uint32_t span = (uint32_t)row, lane = threadIdx.x & 31, warp = threadIdx.x / 32, share = a.span / kWarps;
  const uint64_t c0 = slice * 32 * N, c = c0 + emb_first<N, VEC>();
  float4* const heads = reinterpret_cast<float4*>(flight) + lane * (N / 4);  // of warp w: + w * 8 N float4s
  uint8_t* const rows = flight + kWarps * 32 * N * 4;
  uint8_t* const mine = rows + warp * (kFlight * kSlot);
  const auto tails = [&](uint32_t w) { return reinterpret_cast<float4*>(rows + w * (kFlight * kSlot)) + lane * (N / 4); };
  const auto put = [&](float4* to, const float (&x)[N]) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) to[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
  };
  const auto add = [&](const float4* from, float (&x)[N]) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) x[4 * q] += from[q].x, x[4 * q + 1] += from[q].y, x[4 * q + 2] += from[q].z, x[4 * q + 3] += from[q].w;
  };
  const uint64_t p0 = (uint64_t)span * a.span + warp * share;
  const uint32_t none = (uint32_t)a.vocab;  // of the tokens that do not count, behind all others
  // lane l has place p0 + l, at most 32 of them
  const uint64_t p = p0 + lane;
  const bool here = lane < share && p < a.rows;
  const uint32_t key = here ? keys[p] : none, next = here && p + 1 < a.rows ? keys[p + 1] : none, place = here ? places[p] : 0;
  const uint32_t before = p0 && p0 <= a.rows ? keys[p0 - 1] : none;
  const uint32_t count = __popc(__ballot_sync(0xffffffffu, key != none)), ends = __ballot_sync(0xffffffffu, next != key);
  // the lane's place's rows, handed to all lanes when it is their turn
  const uint64_t my_source = reinterpret_cast<uint64_t>(a.dy) + (uint64_t)place * a.dy_stride * From::es;
  const uint64_t my_target = reinterpret_cast<uint64_t>(a.dtable) + (uint64_t)key * a.table_stride * To::es;
  const auto source = [&](uint32_t i) { return reinterpret_cast<const void*>(__shfl_sync(0xffffffffu, my_source, i)); };
  const auto target = [&](uint32_t i) { return reinterpret_cast<char*>(__shfl_sync(0xffffffffu, my_target, i)); };
  const auto ask = [&](uint32_t i) {
    if (i < count) {
      uint8_t* const slot = mine + i % kFlight * kSlot;
      From::copy(slot, source(i), c0, a.cols);
      if (ADD && (ends >> i & 1)) To::copy(slot + From::kBytes, target(i), c0, a.cols);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (uint32_t i = 0; i < kFlight; ++i) ask(i);
  uint32_t what = 0;
  if (count) {
    const uint32_t key0 = __shfl_sync(0xffffffffu, key, 0), key1 = __shfl_sync(0xffffffffu, key, count - 1);
    bool inside = p0 == 0 || before != key0;  // whether the places summed now start in this share
    // the spans over which the first and the last places reach, asked for while the rows are on their way
    if (warp == 0 && !inside) {
      const uint32_t f = emb_first_span(a, keys, span, key0);
      if (lane == 0) first_span = f;
    }
    if (warp == kWarps - 1 && count == share && !(ends >> (count - 1) & 1)) {
      const uint32_t l = emb_last_span(a, keys, span, key1);
      if (lane == 0) last_span = l;
    }
    float sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = 0.0f;
#pragma unroll 1
    for (uint32_t i = 0; i < count; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kFlight - 1) : "memory");
      if (!VEC) __syncwarp();
      const uint8_t* const slot = mine + i % kFlight * kSlot;
      float x[N];
      From::read(slot, VEC ? nullptr : source(i), c0, x);
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] += x[k];
      if (ends >> i & 1) {
        if (inside) {
          char* const to = target(i);
          if (ADD) To::read(slot + From::kBytes, to, c0, x);
          emb_finish<WDT, N, VEC, ADD>(a, to, c, sum, x);
        } else {
          put(heads + warp * (8 * N), sum);
          what = HEAD | HEAD_ENDS;
        }
        inside = true;
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] = 0.0f;
      }
      if (!VEC) __syncwarp();
      ask(i + kFlight);
    }
    __syncwarp();  // a tail takes the place of rows that other lanes have read
    if (!(ends >> (count - 1) & 1)) {  // the last places go on
      put(inside ? tails(warp) : heads + warp * (8 * N), sum);
      what |= inside ? TAIL : HEAD;
    }
    if (lane == 0) keys_left[warp] = what & TAIL ? key1 : key0;
  }
  if (lane == 0) left[warp] = what;
  __syncthreads();
  // from share to share: what starts in this one, and in the first also what comes from the span before
  for (uint32_t from_before = 0; from_before < 2; ++from_before) {
    if (from_before ? warp != 0 || !(left[0] & HEAD) : !(what & TAIL)) continue;
    float sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = 0.0f;
    uint32_t w = from_before ? 0 : warp + 1, token = keys_left[warp];
    if (from_before) {
      if (what & TAIL) token = __shfl_sync(0xffffffffu, key, 0);
    } else {
      add(tails(warp), sum);
    }
    bool end = false;
    for (; w < kWarps && !end; ++w) {
      add(heads + w * (8 * N), sum);
      end = left[w] & HEAD_ENDS;
    }
    if (end && !from_before) {
      char* const to = static_cast<char*>(a.dtable) + (uint64_t)token * a.table_stride * To::es;
      float old[N];
      EmbRaw<WDT, N, VEC> raw;
      if (ADD) raw.load(to, c, a.cols);
#pragma unroll
      for (int k = 0; k < N; ++k) old[k] = ADD ? raw.at(k) : 0.0f;
      emb_finish<WDT, N, VEC, ADD>(a, to, c, sum, old);
    } else {
      put(reinterpret_cast<float4*>(a.partial + (((uint64_t)span * 2 + (from_before ? 0 : 1)) * a.across + slice) * 32 * N + lane * N), sum);
      emb_join<WDT, N, VEC, ADD>(a, from_before ? first_span : span, end ? span : last_span, (uint32_t)slice, token);
    }
  }
}

}  // namespace ra
