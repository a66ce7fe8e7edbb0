// Programmatic dependent launch of the block operators' kernels: a kernel may be
// set up on the GPU while the one before it in its stream finishes, and waits
// for that one's completion (and its writes) before it touches memory.
#pragma once

#include <cuda_runtime.h>

namespace convrot {

// First statement of every kernel launched with launch_after(): lets the next
// kernel be set up, then waits for the previous one.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches `k`; cluster > 1: CTAs per cluster.
template <typename Kern, typename... Args>
[[maybe_unused]] static cudaError_t launch_after(Kern k, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                                                 Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace convrot
