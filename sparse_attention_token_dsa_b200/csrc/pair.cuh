// pair.cuh — building blocks of kernels whose CTAs work in pairs (clusters of two
// that share one matrix instruction): cluster addresses and barriers, tcgen05 with
// cta_group::2.
#pragma once
#include "operand.cuh"

namespace dsa {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
}
// Cluster address of `p` (a place in this CTA's shared memory) in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Arrive on a barrier of the cluster.  Relaxed, so only for what announces no shared memory:
// TMEM read back, which tcgen05.fence orders with the arrival.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// Arrive for shared memory of this CTA that the pair's matrix instructions may read: written by
// threads (which have fenced it for the async proxy and met the arriving one since) or by TMA
// (complete on a barrier that this thread has seen).  The release and its counterpart behind
// the wait, pair_acquire, order shared memory alone.  A release of all memory over the cluster
// holds its thread for hundreds of clocks: with it a prompt chunk took 1.42 ms where it takes
// 1.00 (and 0.99 with nothing ordered), the 128K decode batch 1.64 for 1.33, 24 ragged
// sequences of e4m3 rows 153 us for 118.
__device__ __forceinline__ void pair_publish(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_cluster(bar);
}
__device__ __forceinline__ void pair_acquire() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// Whether a phase is complete, without waiting for it (mbar_try_wait may suspend its thread
// for up to 20 us, too long for a look ahead that nobody has to wait for: it held back the
// matrix instructions behind it, the last ones of a cluster for all that time, and a batch
// of 24 ragged sequences took 131 us where it took 104).  Relaxed, over the cluster.
__device__ __forceinline__ bool mbar_seen(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What the waits of a CTA share: whether one of them has given up, and how long each may last.
struct WaitLimit {
  int32_t abort;
  int32_t kilocycles;      // SM clocks / 1024
};
__device__ __forceinline__ long long wait_cycles(volatile WaitLimit* w) {
  return (long long)w->kilocycles << 10;
}
// As mbar_wait, with the polling out of line: a kernel with a role for every warp has
// dozens of waits, and inlined polls pushed its loops out of the instruction cache.
template <bool CLUSTER>
__device__ __noinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile WaitLimit* limit,
                                       int32_t* status, int where) {
  return mbar_wait<CLUSTER>(bar, parity, &limit->abort, status, where, wait_cycles(limit));
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_far(uint64_t* bar, uint32_t parity,
                                              volatile WaitLimit* limit, int32_t* status,
                                              int where) {
  return mbar_try_wait<CLUSTER>(bar, parity) ||
         mbar_poll<CLUSTER>(bar, parity, limit, status, where);
}

// ------------------------------------------------------------ cta_group::2 --
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t addr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(ncols)
               : "memory");
}
// One arrival on `bar` (at the same place in both CTAs) when every MMA this thread has
// issued so far is complete.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// One lane of a converged warp.  Matrix instructions stand under this and not under a
// test of the lane's number: their operands then stay in uniform registers (43 against 77
// clocks from one MMA to the next, N = 128).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}
// bf16 MMA of the pair: M = 128 rows, 64 from each CTA's A tile; N columns, half from
// each CTA's B tile; the descriptors name the same places in both CTAs.  CTA c's TMEM
// receives its own 64 rows: lanes 0-63 hold columns 0 .. N/2 - 1, lanes 64-127 columns
// N/2 .. N - 1 of the same rows.
__device__ __forceinline__ void pair_mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

}  // namespace dsa
