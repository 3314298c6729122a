// paged_pair_parts.cuh -- what the chunk kernels on pairs of CTAs share
// (paged_pair.cu, paged4_pair.cu): barriers and arrivals across a cluster of two.
#pragma once

#include "paged_chunk_parts.cuh"

namespace spark {
namespace chunk {

constexpr int kPairTokens = 2 * paged::kChunkTokens;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// every thread of both CTAs
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// this shared-memory address in rank 0, and an arrival there
__device__ __forceinline__ uint32_t in_rank0(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
// ... releasing what this thread wrote to memory,
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// ... or without: what the barrier is about lies in tensor memory, which
// tcgen05's own fences order (a release over the cluster took 1000 to 1400
// cycles of a 3400-cycle tile here)
__device__ __forceinline__ void arrive_tmem_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// a wait, bounded like every other, for what the other CTA did
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort) {
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (done()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0;; ++it) {
    if (done()) return true;
    if ((it & 63u) == 63u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
  }
}

}  // namespace chunk
}  // namespace spark
