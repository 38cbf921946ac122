// tcgen05.cuh -- inline-PTX helpers for the fifth-generation tensor cores of
// sm_103a: tensor memory, matrix instructions on shared-memory operands, and the
// tiled TMA loads that feed them, for a pair of CTAs that work on one tile
// (cta_group::2; the pair is a cluster of two).
#pragma once

#include <cstdint>

#include <cuda.h>

#include "ptx.cuh"

namespace moe {

// mbar_wait for waits on the critical path: polls a while before it reads the (slow) global
// timer that bounds the wait.
template <bool kCluster = false>
__device__ __forceinline__ bool stage_wait(uint32_t bar, uint32_t parity, int32_t* err) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i)
    if (mbar_try_wait<kCluster>(bar, parity)) return true;
  return mbar_wait<kCluster>(bar, parity, err);
}
template <bool kCluster = false>
__device__ __forceinline__ bool stage_wait_warp(uint32_t bar, uint32_t parity, int32_t* err) {
  // one lane polls for a converged warp; the warp's barrier orders the others' accesses after what
  // that lane has seen (a shuffle alone orders no memory)
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = stage_wait<kCluster>(bar, parity, err);
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// True for one lane of a converged warp.  Unlike lane == 0 the compiler knows that a branch on
// it runs one thread, and keeps the operands of TMA and matrix instructions there in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// The registers of a thread, changed by all warps of a warpgroup.  What some take must be no more
// than the others of the block release.
template <int kCount>
__device__ __forceinline__ void registers_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCount));
}
template <int kCount>
__device__ __forceinline__ void registers_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kCount));
}

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {  // a whole warp of each CTA
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {  // the warps that allocated
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

// 16 lanes x 32 columns of fp32: with g = lane / 4 and q = 2 (lane % 4) of the thread,
// v[4 i .. 4 i + 3] are (g, 8 i + q), (g, 8 i + q + 1), (g + 8, 8 i + q), (g + 8, 8 i + q + 1).
// The warp's quarter of the 128 lanes holds two such halves.
__device__ __forceinline__ void tmem_load_16x32(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Four 8 x 8 blocks of 16-bit values, transposed on the way: element (g, q) of a thread's pair
// (g = lane / 4, q = 2 (lane % 4)) lies at place g of memory row q.  Lane 8 b + j gives the
// address of row j of block b.
__device__ __forceinline__ void store_blocks_transposed(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void load_blocks_transposed(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// ------------------------------------------------------- matrix instructions

// Shared-memory operand in the 128-byte swizzle of a TMA box 128 bytes wide (64
// elements of 16 bits), base 1024-byte aligned.
//   contraction contiguous: rows of 128 bytes, groups of 8 rows 1024 bytes apart;
//     16 contraction elements further on are 32 bytes
//   contraction strided (the other extent contiguous): rows of one contraction index,
//     groups of 8 of them 1024 bytes apart, boxes of 64 contiguous elements `box_bytes`
//     apart; 16 contraction elements further on are 2048 bytes
constexpr uint64_t kDescBase = (uint64_t(1) << 46) | (uint64_t(2) << 61) | (uint64_t(1024 >> 4) << 32);
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t box_bytes) {
  return kDescBase | (uint64_t(box_bytes >> 4) << 16) | uint64_t((addr & 0x3ffffu) >> 4);
}

// Instruction word of kind::f16: fp32 accumulators, both operands fp16 or both bf16,
// *_strided where the operand's contraction index is the strided one; N / 8 goes to bit 17.
inline uint32_t mma_word(bool bf16, bool a_strided, bool b_strided, int m) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_strided ? 1u << 15 : 0u) | (b_strided ? 1u << 16 : 0u) |
         (uint32_t(m >> 4) << 24);
}

// D (+)= A B over 16 contraction elements, by one thread of the pair's first CTA: each CTA holds
// its 128 rows of A and D, and half of B's columns, at the same shared-memory addresses.
__device__ __forceinline__ void mma_f16(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t word, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          tmem_d),
      "l"(a), "l"(b), "r"(word), "r"(accumulate)
      : "memory");
}

// Arrives on the barrier in the cluster's CTAs of the mask when the thread's matrix instructions so
// far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t ctas) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(ctas))
      : "memory");
}

// ----------------------------------------------------------- tiled TMA loads
//
// The bytes are counted on a barrier of the pair's first CTA (`bar` is its cluster address).

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
      : "memory");
}
// For a CTA on its own.
__device__ __forceinline__ void tma_load_5d_single(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                                   int v, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
      : "memory");
}

// Tiled store from shared memory, in the issuing thread's bulk group; elements outside the map
// are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's stores have read their shared memory / are done.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without an order of memory accesses.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// The address in the cluster's shared window of `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 bytes to another CTA's shared memory, counted on a barrier there (both cluster addresses).
__device__ __forceinline__ void store_async_16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void store_async_4(uint32_t addr, float x, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(x)), "r"(bar)
               : "memory");
}
// Arrives on a barrier of either CTA (a cluster address) once the thread is done with tensor memory:
// its loads are complete and fenced (tcgen05_fence_before), and nothing that it wrote is read by who
// waits.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The same after writes of the warp to its CTA's shared memory, which instructions of the waiting
// thread read: a release of those writes alone.  A release of all memory for the cluster costs the
// weight gradient of 16384 rows over 128 experts, 2048 x 1408, 29 us more.
__device__ __forceinline__ void mbar_arrive_cluster_shared(uint32_t addr) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_cluster_relaxed(addr);
}

}  // namespace moe
