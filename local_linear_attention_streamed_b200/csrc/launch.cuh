// Launches that overlap the set-up of a kernel with the end of the one before it.
#pragma once

#include <cuda_runtime.h>

namespace plx {

// Until the kernels before this one in the stream have ended and their writes
// are visible; called before any access to memory that they may touch (through
// pointers without __restrict__, whose loads might be moved above it).
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on the next kernel in the stream may be set up, if it was launched
// by launch_dependent (and calls grid_dep_wait).
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The kernel has to call grid_dep_wait.  cluster: CTAs of a cluster along x, 1 for none.
template <typename Kern, typename... Args>
cudaError_t launch_dependent(Kern kern, dim3 grid, unsigned block, size_t smem, int cluster, cudaStream_t st,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace plx
