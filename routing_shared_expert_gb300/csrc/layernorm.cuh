// Normalisation of rows, LAYER or RMS: what the forward and the backward pass share.
//
//   h = x + r,  mean = sum h / d,  rstd = (sum (h - mean)^2 / d + eps)^(-1/2),  y = (h - mean) rstd w + b
//   xhat = (h - mean) rstd,  g = dy w,
//   dx = rstd (g - sum g / d - xhat sum (g xhat) / d) + dsum,  dw = sum_t dy xhat,  db = sum_t dy
// (RMS: mean = 0, no sum g).  The variance is taken from deviations, never as E h^2 - mean^2.
#pragma once

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "row_reduce.cuh"
#include "vec8.cuh"

namespace moe {

struct NormArgs {
  const void* x;        // h in the backward pass
  const void* r;        // residual, or dsum
  const void* w;
  const void* b;
  void* s;              // sum, or dx
  void* y;              // dy in the backward pass (read only)
  float* mean;
  float* rstd;
  float* partial;       // [slots][2][d]
  float* dw;
  float* db;
  int64_t T, ldx, ldr, lds, ldy;
  int32_t d, slots;
  float eps;
  int32_t rms, w_dtype;
  int32_t lanes;        // of a row (SPLIT)
  int32_t stages;       // rows on their way, 2 to 4
};

__device__ __forceinline__ float load_param(const void* p, int32_t dtype, int32_t c, float none) {
  if (!p) return none;
  return dtype == MOE_F32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const __nv_bfloat16*>(p)[c]);
}

// The gradients (layernorm_grad.cu).
cudaError_t launch_layernorm_backward(const NormArgs& a, const moe_layernorm_config& c, cudaStream_t s);

// --------------------------------------------------------------- rows in groups --
// Rows whose operands all start at the same place within a group of eight elements (aligned
// tensors with one width or stride, odd ones included): a thread takes P groups of eight.  A row
// that starts `phase` elements into a group has two end groups that are not whole.  The rows of a
// CTA are gridDim.x apart, a multiple of eight unless the stride is one, so that the phase is the same
// for all of them; the parameters lie in shared memory at that phase.  SPLIT: `lanes` lanes of a warp
// (a power of two) take a row and the CTA 256 / lanes rows at once, with no barrier; else the whole CTA
// takes one.
//
// Each thread copies its own groups of the next rows asynchronously into its own slots of a ring in
// shared memory, a.stages rows ahead: the bytes on their way do not depend on registers, and the
// ring needs no barrier.

// Values 8 q .. 8 q + 7 of a parameter in shared memory: the lower and the upper half of all groups
// apart, so that neighbouring lanes' 16-byte reads are neighbours.
__device__ __forceinline__ void param8(const float* p, int groups, int q, float (&v)[8]) {
  const float4 lo = reinterpret_cast<const float4*>(p)[q], hi = reinterpret_cast<const float4*>(p)[groups + q];
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}
__device__ __forceinline__ void stage_param(float* dst, const void* src, int32_t dtype, int groups, int phase, int d) {
  for (int i = threadIdx.x; i < 8 * groups; i += blockDim.x) {
    const int c = i - phase, q = i >> 3, j = i & 7;
    dst[(j >> 2) * 4 * groups + 4 * q + (j & 3)] = c >= 0 && c < d ? load_param(src, dtype, c, 0.f) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ int phase_of(const T* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7;
}
__device__ __forceinline__ void wait_stage(int stages) {   // the oldest of `stages` copies has landed
  if (stages == 2) cp_async_wait<1>();
  else if (stages == 3) cp_async_wait<2>();
  else cp_async_wait<3>();
}

template <bool SPLIT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (&part)[2][N * 32], int& turn, int lanes) {
  if (SPLIT) {
    for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else {
    block_sum<N>(v, part[turn]);
    turn ^= 1;
  }
}

// ------------------------------------------------------------------ launch plan --

constexpr int kMaxGroups = 2048;                  // of a row: 512 threads of four
constexpr size_t kSharedPerSm = 227 * 1024;

// How rows are taken in groups of eight, if they can be.
struct Plan {
  int groups_per_thread = 0;   // 0: any layout
  int lanes = 0, threads = 0, stages = 0;
  bool split = false;
  unsigned grid = 0;
  size_t smem = 0;
};

template <typename T>
bool same_phase(const void* p, int64_t ld, int64_t rows, int64_t phase, int64_t ld8) {
  if (!p) return true;
  return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / sizeof(T) & 7) == phase && (rows == 1 || ld % 8 == ld8);
}

// pieces: of 16 bytes, that a group of all operands which are read takes; params: fp32 rows of
// parameters in shared memory; most: CTAs at most; resident: threads of an SM that the kernels'
// registers leave room for, with two groups per thread.
template <typename X, typename S, typename Y>
Plan make_plan(const NormArgs& a, int pieces, int params, int64_t most, int resident) {
  Plan p;
  const int64_t phase = reinterpret_cast<uintptr_t>(a.x) / sizeof(X) & 7, ld8 = a.ldx % 8;
  const bool ok = same_phase<S>(a.r, a.ldr, a.T, phase, ld8) && same_phase<S>(a.s, a.lds, a.T, phase, ld8) &&
                  same_phase<Y>(a.y, a.ldy, a.T, phase, ld8);
  const bool shifts = ld8 != 0 && a.T > 1;              // the phase differs from row to row
  const int groups = static_cast<int>((a.d + (shifts ? 7 : phase) + 7) / 8);
  if (!ok || groups > kMaxGroups) return p;
  p.split = groups <= 64;
  int per;
  if (p.split) {
    per = groups <= 32 ? 1 : 2;
    p.lanes = 32;
    while (p.lanes / 2 >= groups) p.lanes /= 2;
    p.threads = 256;
  } else {
    per = groups <= 1024 ? 2 : 4;
    p.threads = ((groups + per - 1) / per + 31) / 32 * 32;
    p.lanes = p.threads;
  }
  // as many CTAs to an SM as their registers let in, fewer where their rings would be too short
  const size_t fixed = static_cast<size_t>(p.lanes) * per * 32 * params, stage = static_cast<size_t>(p.threads) * per * 16 * pieces;
  int per_sm = std::max(1, (per == 4 ? 512 : resident) / p.threads);
  for (;; --per_sm) {
    for (p.stages = 4; p.stages > 2 && per_sm * (fixed + p.stages * stage + 2048) > kSharedPerSm;) --p.stages;
    if (per_sm <= 1 || per_sm * (fixed + p.stages * stage + 2048) <= kSharedPerSm) break;
  }
  p.smem = fixed + p.stages * stage;
  if (p.smem + 2048 > kSharedPerSm) return p;
  p.groups_per_thread = per;
  const int64_t at_once = p.split ? 256 / p.lanes : 1;
  int64_t ctas = std::min({(a.T + at_once - 1) / at_once, most, static_cast<int64_t>(per_sm) * device_sm_count()});
  if (shifts && (p.split || ctas < a.T)) ctas = std::max<int64_t>(8, ctas / 8 * 8);
  p.grid = static_cast<unsigned>(ctas);
  return p;
}

// The limit of a kernel's shared memory, raised where the plan needs more than every kernel has (48 KB, the
// kernel's own static arrays among them).
template <typename F>
cudaError_t allow_smem(F f, size_t bytes) {
  return bytes > 47 * 1024 ? set_smem_once(reinterpret_cast<const void*>(f), bytes) : cudaSuccess;
}

}  // namespace moe
