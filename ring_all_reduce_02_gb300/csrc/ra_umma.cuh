// The instructions of a tensor-core product on sm_103a: tiles brought in by the
// Tensor Memory Accelerator, tcgen05.mma over a pair of CTAs, accumulators in
// tensor memory. Thin wrappers; every wait is bounded.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "ra_bulk.cuh"

namespace ra {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// True in one lane, the same one each time, of a warp that comes here together.
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}
// A value that is the same in all lanes, so that the compiler keeps what follows from it in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared memory p in the pair's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_address(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// An arrival at a barrier of either CTA of a pair that only says that something has been read. It is relaxed, and by itself
// would not stay behind a read of shared memory that has been issued but not answered. What has been read has to have reached
// registers, in all lanes whose reading it speaks for: a tile's words have gone through shuffles of the whole warp by then
// (which take the values, not the addresses), and accumulators are waited for by tcgen05.wait::ld and handed over by a tcgen05
// fence. (One with release of the cluster's scope waits for the thread's stores to global memory, half a microsecond and more.)
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// 32 bytes to either CTA of a pair, and the arrival at its barrier that says so.
__device__ __forceinline__ void store_pair(uint32_t cluster_addr, const uint32_t (&w)[8], uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 32;" ::"r"(cluster_bar) : "memory");
#pragma unroll
  for (int i = 0; i < 8; i += 4)
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr + 4 * i),
                 "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(cluster_bar)
                 : "memory");
}

constexpr uint64_t kPairWaitNs = 4000000000ull;  // 4 s: more than any tile takes
// Whether the phase of a barrier has ended. An acquire of the CTA's scope does for arrivals from the other one: what is read
// behind it lies in this CTA's shared memory or in tensor memory (one of the cluster's scope also empties the L1 cache, at
// 0.3 us).
__device__ __forceinline__ bool mbar_try_pair(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// As mbar_wait, for `limit` ns at most, by one thread. Where it gives up, `what` says in *dead which wait did; where the CTA
// already has, it gives up at once.
__device__ __forceinline__ bool mbar_wait_pair(uint64_t* bar, uint32_t parity, volatile int* dead, int what, uint64_t limit) {
  uint64_t start = 0;
  while (!mbar_try_pair(bar, parity)) {
    if (*dead) return false;
    const uint64_t now = global_ns();
    if (start == 0) start = now;
    if (now - start > limit) {
      *dead = what;
      return false;
    }
  }
  return true;
}
// The same by a whole warp, whose lanes all have the same answer: a lane may see the phase end when another one sees that
// the CTA has given up, and what follows a wait (shuffles, tensor memory) takes all 32.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* dead, int what, uint64_t limit) {
  uint64_t start = 0;
  while (!__all_sync(0xffffffffu, mbar_try_pair(bar, parity))) {
    const uint64_t now = global_ns();
    if (start == 0) start = now;
    if (__any_sync(0xffffffffu, *dead != 0 || now - start > limit)) {
      if ((threadIdx.x & 31) == 0 && *dead == 0) *dead = what;
      __syncwarp();
      return false;
    }
  }
  return true;
}

// A box of a two-dimensional tensor map into this CTA's shared memory; its bytes are counted by the barrier at
// `cluster_bar`, in either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}
// The same of a three-dimensional one.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}
// A box on its way into L2.
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
// A box out of shared memory, by one thread; the waits are for what that thread has stored: until shared memory has been
// read, and until all is written.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* from, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\tcp.async.bulk.commit_group;" ::"l"(map),
               "r"(x), "r"(y), "r"(smem_u32(from))
               : "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_stores_written() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory ---------------------------------------------------------------
// One warp of each CTA of the pair; the address is written to *slot.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t address, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(address), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 columns of the warp's 32 lanes: lane l's into its x[0..31].
__device__ __forceinline__ void tmem_load32(uint32_t address, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]),
        "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]),
        "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]),
        "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
      : "r"(address));
}

// ---- products ----------------------------------------------------------------------
// Operand tiles lie in shared memory as boxes of 64 x 64 16-bit elements, rows of 128 bytes with their 16-byte lines
// swizzled (line l of row r at l ^ (r % 8)), 8192 bytes a box. An operand whose rows run along the summed dimension
// ("summed inner") has its boxes one below the other: 8-row groups are 1024 bytes apart. One whose rows run along its
// own dimension ("own inner") has a box for every 64 of them: boxes are 8192 bytes apart, groups of 8 summed
// elements 1024.
constexpr uint32_t kBoxBytes = 8192;
__device__ __forceinline__ uint64_t umma_descriptor(uint32_t smem_addr, bool own_inner) {
  const uint64_t groups = 1024 >> 4, boxes = own_inner ? kBoxBytes >> 4 : 1;
  return (uint64_t)((smem_addr & 0x3ffffu) >> 4) | boxes << 16 | groups << 32 | 1ull << 46 | 2ull << 61;
}
// How far 16 summed elements lie apart, in the descriptor's units of 16 bytes.
__device__ __forceinline__ uint32_t umma_step(bool own_inner) { return own_inner ? 16 * 128 / 16 : 32 / 16; }
// fp32 accumulators, 16-bit operands (bf16 or fp16), 256 x n.
__device__ __forceinline__ uint32_t umma_instruction(bool bf16, bool a_own_inner, bool b_own_inner, uint32_t n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_own_inner ? 1u << 15 : 0u) | (b_own_inner ? 1u << 16 : 0u) | (n >> 3) << 17 |
         (256u >> 4) << 24;
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
      "r"(instruction), "r"(add ? 1u : 0u)
      : "memory");
}
// Arrives at the barrier at `bar`'s place in both CTAs once every product issued so far is done.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}

}  // namespace ra
