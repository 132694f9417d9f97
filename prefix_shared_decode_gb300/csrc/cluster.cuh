// What the kernels that rank or choose by clusters share: the clusters' shared
// memories, and floats as integers of the same order.
#pragma once

#include "device.cuh"

namespace ca {
namespace dev {

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_peer(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t order_key(float x) {   // monotone; 0 for a NaN, at most 0xff800000
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);           // -0 counts as 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace dev
}  // namespace ca
