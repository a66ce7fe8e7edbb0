// Programmatic dependent launch of the block operators' kernels: a kernel may be
// set up on the GPU while the one before it in its stream finishes, and waits
// for that one's completion (and its writes) before it touches memory.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace convrot {

// First statement of every kernel launched with launch_after(): lets the next
// kernel be set up, then waits for the previous one.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Loads for these kernels.  Each triggers before it waits, so a kernel's life
// overlaps that of the one that writes its operands, and of the one before that,
// which may read the same addresses on the same SM: the non-coherent path
// (ld.global.nc, __ldg, const __restrict__ parameters), for memory that nobody
// writes while the kernel lives, could return the old values, and the compiler
// may move such a load ahead of the wait.  These are plain loads, issued where
// they stand, and take no longer (19989 x 5376, K = 14336, gate and residual
// 1761 us; one token x 5376 x 21504 in S8 codes 22.4; norm 125.4; rotary 176.3).
__device__ __forceinline__ float load_global(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load_global(const float4* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_global(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int32_t load_global(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ double load_global(const double* p) {
  double v;
  asm volatile("ld.global.f64 %0, [%1];" : "=d"(v) : "l"(p));
  return v;
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
