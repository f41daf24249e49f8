// Sums over the threads of a CTA that share a row.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the whole CTA, the same in every thread.  `part` holds N * 32 floats; the
// callers alternate between two such buffers, so that one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? part[i * 32 + lane] : 0.f);
}

}  // namespace moe
