// Inline PTX of the int8 GEMM: tcgen05 MMAs of kind i8 by one CTA and by a CTA pair, the pair's TMEM
// allocation, copies and commits, and the thread-block cluster primitives.
#pragma once
#include "common.cuh"

namespace svdq {

// Instruction descriptor, kind::i8: A, B signed 8-bit (K-major), D = s32 (wrapping), M x N, K = 32.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D(tmem) (+)= A(smem) x B(smem)^T on one CTA.
SVDQ_DEV void tc_mma_i8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same by a CTA pair: each CTA holds half of A's rows and half of B's, and its rows of D.
SVDQ_DEV void tc_mma_i8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// TMEM of a pair: one warp of each CTA takes part.
SVDQ_DEV void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
}
SVDQ_DEV void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
SVDQ_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrive once on the barrier at `bar`'s offset in both CTAs of the pair when every tcgen05 operation this
// thread issued before it has completed.
SVDQ_DEV void tc_commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// ------------------------------------------------------- warp-uniform issuing ---
// Copies and MMAs take their operands from uniform registers.  Where the compiler can prove a role's
// control flow and operands uniform over the warp, an issue takes a few cycles; under a branch on the lane
// it wraps each one in a loop over the active lanes (measured: 70 cycles an MMA, 600 a ring stage).  So a
// role's whole warp walks its loop, values that come from shared memory or special registers pass through
// warp_uniform, and only the issue itself is under elect_one().
SVDQ_DEV uint32_t warp_uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
SVDQ_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// mbar_wait_spin by a whole warp, with one answer for all its lanes.
SVDQ_DEV bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort, unsigned site) {
  const uint32_t a = smem_u32(bar);
  if (__all_sync(0xFFFFFFFFu, mbar_test_wait(a, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 0;; ++n) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(a, parity))) return true;
    if ((n & 15u) == 15u && __any_sync(0xFFFFFFFFu, *abort != 0 || globaltimer_ns() - t0 > timeout_ns)) {
      if (elect_one() && !*abort) {
        *abort = 1;
        report_timeout(site);
      }
      __syncwarp();
      return false;
    }
  }
}

// ---------------------------------------------------------------- clusters ---
SVDQ_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared address of `addr` in CTA `rank` of the cluster.
SVDQ_DEV uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// All threads of all CTAs of the cluster; writes before it are visible after it.
SVDQ_DEV void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
SVDQ_DEV int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
SVDQ_DEV float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
SVDQ_DEV void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Makes this thread's stores to shared memory visible to copies and MMAs issued after the next barrier.
SVDQ_DEV void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 2-D tiled load into this CTA's shared memory, completion counted on a barrier of the pair (a
// shared::cluster address: the leader's).
SVDQ_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

}  // namespace svdq
