// Clusters of CTAs: their barrier, and words into one another's shared memory.
#pragma once

#include "tc_ptx.cuh"

namespace tq {
namespace serve {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// A shared-memory address of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(tc::smem_addr(p)), "r"(rank));
    return r;
}
// 16 or 8 bytes into another CTA's shared memory.
__device__ __forceinline__ void send(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void send(uint32_t to, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};\n" ::"r"(to), "r"(a), "r"(b) : "memory");
}
// The cluster's barrier: every thread of it arrives, and waits once for each arrival. What was written before an arrival is seen behind
// the wait, in all CTAs. (The hardware's own: it ends as soon as all threads have arrived, or ended.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory"); }

}  // namespace serve
}  // namespace tq
