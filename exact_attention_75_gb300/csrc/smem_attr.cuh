// Kernel launches: opting into more than 48 KB of dynamic shared memory, and
// launching as a programmatic dependent.
//
// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) is a setting of the
// current device's context, so a process that calls on device 0 and then on
// device 1 must set it on both.  Each launch site keeps one flag per device
// ordinal (an array of its own: the flag belongs to one kernel instantiation)
// and sets the attribute the first time it launches on a device.  The flags
// are atomics because the C ABI may be called from several host threads;
// setting the attribute twice is harmless.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace attn {

constexpr int kMaxAttrDevices = 64;

using DeviceFlags = std::atomic<bool>[kMaxAttrDevices];

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

template <typename Kern>
cudaError_t ensure_dyn_smem(Kern kern, int bytes, DeviceFlags& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < kMaxAttrDevices;
  if (tracked && configured[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && tracked) configured[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace attn
