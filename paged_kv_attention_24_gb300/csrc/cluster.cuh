// Blocks of a cluster: their barrier and each other's shared memory.
#pragma once

#include <stdint.h>

namespace msgl {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The barrier's two halves, by every thread.  What was written before arriving (here and in other blocks' shared memory)
// is there after waiting.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Arriving with nothing written: a block has to run before another writes into its shared memory.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }

// The address of p (in shared memory) in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_address(const void *p, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return at;
}

}  // namespace msgl
