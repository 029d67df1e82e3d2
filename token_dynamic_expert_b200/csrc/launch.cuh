// launch.cuh -- the launch of the 8-bit layer's kernels.
//
// They follow one another in a stream, most of them shorter than a launch takes,
// so each is launched with programmatic stream serialisation: its CTAs may be
// scheduled while the kernel before it ends.  begin_overlapped(), which every
// thread of such a kernel calls before its first access to global memory, lets
// the next launch be scheduled and waits until the kernel before has completed
// and its memory is visible, so stream order holds for every argument.
#pragma once

#include "ace_common.cuh"
#include "ace_internal.h"

namespace ace {

__device__ __forceinline__ void begin_overlapped() {
  allow_dependent_launch();
  grid_dependency_wait();
}

// kernel<<<grid, block, smem, s>>>(args...), in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block,
                              unsigned cluster, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace ace
