// Launches that may begin under the one before them in their stream (host).
#pragma once

#include <cuda_runtime.h>

namespace moe {

// The kernel begins its set-up under the previous launch and waits (wait_for_previous) before it looks at
// any operand.
template <typename... A>
cudaError_t launch_over(void (*f)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... a) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(static_cast<unsigned>(threads));
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, f, a...);
}

}  // namespace moe
