// cluster.cuh -- thread-block clusters: rank, barrier, and words of the other
// CTAs' shared memory.
#pragma once

#include "common.cuh"

namespace smoe {

__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size()
{
    unsigned n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// The barrier of all threads of the cluster: what they wrote before it, to
// shared or global memory, is seen behind it.  Every thread calls both halves.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

// Stores v to the word that `own` is in the shared memory of CTA `rank`, which
// must have started (a barrier before) and not ended (a barrier after).
__device__ __forceinline__ void store_to_rank(int *own, unsigned rank, int v)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(own)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

}  // namespace smoe
