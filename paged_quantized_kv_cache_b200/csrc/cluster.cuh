// cluster.cuh -- thread-block clusters: their barrier and distributed shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pqkv {

// Barrier of all threads of the cluster; shared-memory writes before it are
// visible to the peers behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Loads from the shared memory of the cluster's CTA `rank`, at the address that
// `addr` has in this CTA's.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(peer_addr(addr, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_addr(addr, rank))
               : "memory");
  return v;
}

}  // namespace pqkv
