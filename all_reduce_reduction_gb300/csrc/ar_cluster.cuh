// What the layer operators' kernels that run in thread-block clusters share.
#pragma once

#include <stdint.h>

namespace ar {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Barrier of all threads of the cluster.  The warp is brought together first: the
// .aligned form needs every lane at the same instruction.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word or a binary32 number of CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t ld_peer_u32(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ float ld_peer_f32(const void *p, uint32_t rank) {
    return __uint_as_float(ld_peer_u32(p, rank));
}

}  // namespace ar
