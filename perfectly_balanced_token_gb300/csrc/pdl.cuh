// Launches that overlap the end of the kernel before (programmatic stream serialization): a kernel
// sets itself up, then grid_wait() holds every thread until the kernels before it have ended and
// their writes are there; grid_trigger() lets the next kernel begin in the same way.  Measured between
// dependent kernels of a CUDA graph: 1.6 us less for each.
// Every thread of a kernel launched with launch_after() calls grid_wait() before it touches global
// memory.  (Without that, the kernel after it could run before the one in front of it has ended.)  What it
// then reads may have been written since it began, so it is read by ordinary loads, never by non-coherent
// ones (__ldg, or a parameter that is const and __restrict__).
#pragma once

#include <cuda_runtime.h>

namespace moonep {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                                cudaStream_t st, unsigned cluster, A... given) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return [&](P... args) {
    void* list[] = {(void*)&args...};
    return cudaLaunchKernelExC(&cfg, (const void*)kernel, list);
  }(given...);
}

}  // namespace moonep
