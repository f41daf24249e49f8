// Launches that may begin under the one before them in their stream (host).
#pragma once

#include <cuda_runtime.h>

namespace moe {

// Launches a kernel that may begin its set-up under the previous one of the stream: it calls
// wait_for_previous() before it touches global memory.  cluster: CTAs per cluster where the kernel
// does not fix them itself.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, int cluster,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The same without clusters.
template <typename... P, typename... A>
cudaError_t launch_over(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, const A&... args) {
  return launch_overlapped(kernel, grid, block, smem, s, 0, args...);
}

}  // namespace moe
