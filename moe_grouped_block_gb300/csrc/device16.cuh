// device16.cuh -- the 16-bit operators' additions to mxg_device.cuh: launches that
// overlap, waits and arrivals across a cluster, tcgen05 and TMA instructions
// issued by one lane of a converged warp.
#pragma once

#include "mxg_device.cuh"

namespace mxg {

// ---------------------------------------------------------------- kernel after kernel
// A kernel that launch_after (host16.h) started beside the one before it:
// wait until that one has finished and its writes are visible.  And, in the one
// before: let the next start to be set up now.
__device__ __forceinline__ void grid_wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- clusters
// mbar_try_wait for a barrier that threads of another CTA of the cluster arrive
// on (acquire at cluster scope).
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// tmem_ld32 with 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Arrive on an mbarrier named by its shared::cluster address, publishing this
// thread's earlier writes to the cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// ---------------------------------------------------------------- one lane of a converged warp
// The forms below are reached by a whole converged warp and executed by the
// lane whose `leader` is set (elect_leader), with no branch around them: 16384 rows
// through 8 experts of 14336 x 4096 took 1300 us with these instructions behind a
// branch on the lane number, 1241 us in this form.
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

// Bounded wait of a whole converged warp; every lane gets the same answer.
// CLUSTER: threads of another CTA arrive on the barrier.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, int32_t* status,
                                               uint64_t timeout_ns = kWaitTimeoutNs) {
  auto ready = [&] {
    const bool r = CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    return __all_sync(0xFFFFFFFFu, r) != 0;
  };
  if (ready()) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 0;; ++it) {
    if (ready()) return true;
    bool late = false;
    if ((it & 15u) == 15u) late = globaltimer() - t0 > timeout_ns;
    if (__any_sync(0xFFFFFFFFu, late)) {
      *abort_flag = 1;
      status_set(status, MXG_DEV_TIMEOUT);
      return false;
    }
    if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) return false;
  }
}

__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx_if(uint32_t bar, uint32_t bytes,
                                                         uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d_if(uint32_t dst, const void* tmap, uint32_t bar,
                                               int32_t c0, int32_t c1, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair_if(uint32_t dst, const void* tmap,
                                                    uint32_t cluster_bar, int32_t c0, int32_t c1,
                                                    uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(tmap), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair_if(uint32_t dst, const void* tmap,
                                                    uint32_t cluster_bar, int32_t c0, int32_t c1,
                                                    int32_t c2, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(tmap), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(c2), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tc_commit_pair_mc_if(uint32_t bar, uint16_t cta_mask,
                                                     uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"(cta_mask), "r"(leader)
      : "memory");
}

// D(tmem) (+)= A(smem) * B(smem)^T, 16-bit operands (the instruction
// descriptor names the type), FP32 accumulation, on the CTA pair.
__device__ __forceinline__ void tc_mma_f16_pair_if(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                   uint32_t idesc, uint32_t accumulate,
                                                   uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

// cluster_sync in two halves, by whole warps
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// fp32 words in shared memory, this CTA's and another one's of the cluster
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- copies
// cp_async_16 past L1, for data that is read once.
__device__ __forceinline__ void cp_async_16_l2(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

}  // namespace mxg
