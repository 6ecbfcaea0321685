// Programmatic dependent launches and thread-block clusters, as the rotary and
// paged kernels use them.  A header of its own: the sources of the dense kernels
// identify their measured DRAM traffic.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace attn {

// Launches a kernel that calls grid_wait() as a programmatic dependent of the
// previous kernel on the stream, in clusters of `cluster` CTAs.
template <typename Kern, typename... Args>
cudaError_t launch_clusters(Kern kern, int cluster, dim3 grid, int threads, int smem,
                            cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename Kern, typename... Args>
cudaError_t launch_dependent(Kern kern, dim3 grid, int threads, int smem, cudaStream_t stream,
                             const Args&... args) {
  return launch_clusters(kern, 1, grid, threads, smem, stream, args...);
}

#ifdef __CUDACC__

// ------------------------------------------------ programmatic dependence ---
// A kernel launched as a programmatic dependent may start before the previous
// kernel of its stream has finished: grid_wait() returns once that one has
// completed and its writes are visible, and comes before the first access to
// memory that another kernel may touch.  grid_release() lets the next
// dependent start its launch.

__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- clusters ---

// Barrier of all threads of the cluster's CTAs; what they wrote to shared
// memory before is visible to cluster_load after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Loads from the shared memory of the cluster's CTA `rank`, at the address
// that `addr` has in this CTA.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float2 cluster_load2(uint32_t addr, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(cluster_addr(addr, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ float4 cluster_load4(uint32_t addr, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(addr, rank))
               : "memory");
  return v;
}

#endif  // __CUDACC__

}  // namespace attn
