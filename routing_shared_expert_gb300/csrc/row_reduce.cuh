// Sums over the threads that share a row.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A barrier of the `threads` threads (whole warps) that name it; 0 is __syncthreads' own.
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of N values over the warps of a team, W at most, the same in every thread.  `part` holds N * W
// floats of the team's own; its calls alternate between two of them, so that one barrier per sum is enough.
template <int N, int W>
__device__ __forceinline__ void team_sum(float (&v)[N], float* part, int warp, int warps, int barrier) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * W + warp] = v[i];
  named_barrier(barrier, warps * 32);
  const int at = warps > 16 ? lane : lane & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = at < warps ? part[i * W + at] : 0.f;
  if (W > 16 && warps > 16)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// The same over the whole CTA of at most 512 threads.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
  team_sum<N, 16>(v, part, threadIdx.x >> 5, blockDim.x >> 5, 0);
}

}  // namespace moe
