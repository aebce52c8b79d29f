// CTA-pair (cta_group::2) building blocks shared by the SM-pair GEMM and the
// grouped products: cluster addressing, remote arrivals, paired TMA loads and
// MMAs (inline PTX, sm_103a).
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "tc_common.cuh"

namespace mg {
namespace tc {

static __device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// shared::cluster address of the same object in CTA `rank` of this cluster
static __device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(smem_u32(p)), "r"(rank));
  return out;
}

// Arrive on a barrier of another CTA of the cluster.  Default semantics
// (release at CTA scope): it signals that this thread's TMEM reads are done
// (tcgen05.wait::ld, then tcgen05.fence::before_thread_sync), and must not
// wait for the thread's global stores to reach cluster scope -- nothing the
// waiting MMA thread reads depends on them.  (With .release.cluster each
// epilogue warp stalled on a memory barrier per tile, holding the
// accumulator until its output stores were acknowledged.)
static __device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Remote arrive that publishes this thread's earlier writes to the cluster.
static __device__ __forceinline__ void mbar_arrive_remote_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA load into this CTA's shared memory whose completion is counted on the
// leader CTA's barrier (cluster address bar_cluster).
static __device__ __forceinline__ void tma_load_2d_to_leader(void* dst, const CUtensorMap* map,
                                                      uint32_t bar_cluster, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}

static __device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

static __device__ __forceinline__ void mma_bf16_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// Arrive on the barrier at this offset in both CTAs once the pair's MMAs issued
// so far have completed.
static __device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

}  // namespace tc
}  // namespace mg
