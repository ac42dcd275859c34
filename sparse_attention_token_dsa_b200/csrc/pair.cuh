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
// Arrive on a barrier of the cluster.  Relaxed: a release over the cluster costs about a
// thousand clocks a call (the attention kernel's 128K decode batch took 5.84 ms with it and
// 1.84 without), and nothing here needs it.  What the arrival announces is either no memory at all (a slot
// read by the tensor core, TMEM read back) or shared memory of the arriving thread's own
// CTA that the async proxy reads: written by TMA and observed on a barrier, or by this
// warp before a proxy fence, which orders it with the async proxy itself.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// Whether a phase is complete, without waiting for it (mbar_try_wait may suspend its thread
// for up to 20 us, too long for a look ahead that nobody has to wait for: it held back the
// matrix instructions behind it, the last ones of a cluster for all that time, and a batch
// of 24 ragged sequences took 131 us where it takes 104).
__device__ __forceinline__ bool mbar_seen(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// As mbar_wait, with the polling out of line: a kernel with a role for every warp has
// dozens of waits, and inlined polls pushed its loops out of the instruction cache.
__device__ __noinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort,
                                       int32_t* status, int where) {
  return mbar_wait(bar, parity, abort, status, where);
}
__device__ __forceinline__ bool mbar_wait_far(uint64_t* bar, uint32_t parity, volatile int* abort,
                                              int32_t* status, int where) {
  return mbar_try_wait(bar, parity) || mbar_poll(bar, parity, abort, status, where);
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
