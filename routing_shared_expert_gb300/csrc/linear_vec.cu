// The dense projection of one to four tokens: y = act(x W^T + b) + r, bound by reading W once.
//
// A warp takes a weight row (or a part of its depth, where the rows alone are too few warps), its
// lanes neighbouring 16-byte pieces, several on their way at a time; the products accumulate in
// fp32 per lane and are added by shuffles, a row's parts in shared memory in a fixed order.  No
// barriers, tensor memory or clusters to set up: a call costs little more than its reads.
#include <algorithm>

#include "activation.cuh"
#include "linear.h"
#include "load_any.cuh"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int DEEP = 4;      // 16-byte pieces of a weight row on their way per lane

struct Args {
  const __nv_bfloat16* x;
  const __nv_bfloat16* W;
  int64_t ldx, ldw, ldr, ldc;
  int32_t N, K, act;
  int32_t split;             // warps of a CTA that share a row: 1, 2, 4 or 8
  const float* bias;
  const void* residual;
  void* pre;
  void* C;
};

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight values from column k on; zeros past K.  VEC: 16-byte aligned rows of a multiple of 8.
template <bool VEC> struct Piece;
template <> struct Piece<true> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int k, int K, const Span&) {
    u = k < K ? *reinterpret_cast<const uint4*>(row + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void take(const __nv_bfloat16*, int, int, float (&v)[8]) const { unpack8(u, v); }
};
template <> struct Piece<false> {
  Raw8 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int k, int K, const Span& span) {
    r = load8_raw(row + k, k < K ? span : Span{1, 0});
  }
  __device__ __forceinline__ void take(const __nv_bfloat16* row, int k, int K, float (&v)[8]) const {
    take8(r, row + k, K - k, v);
  }
};

__device__ __forceinline__ float act_any(float z, int act) {
#define MOE_CALL(ACT) act_value<ACT>(z)
  MOE_DISPATCH_ACT(act, MOE_CALL)
#undef MOE_CALL
}

template <int T, bool VEC, typename OUT>
__global__ void __launch_bounds__(32 * WARPS) linear_vec_kernel(const Args a) {
  __shared__ float s_part[WARPS][T];
  launch_dependents();
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rows = WARPS / a.split;               // of this CTA
  const int part = warp % a.split;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * rows + warp / a.split;
  float acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = 0.f;
  if (f < a.N) {
    const __nv_bfloat16* wr = a.W + f * a.ldw;
    const Span sw = span_of(a.W, a.N, a.ldw, a.K, 2), sx = span_of(a.x, T, a.ldx, a.K, 2);
    // pieces of 256 columns a warp step, the parts of a row in turn
    for (int k0 = part * 256 + lane * 8; k0 < a.K; k0 += a.split * 256 * DEEP) {
      Piece<VEC> w[DEEP];
#pragma unroll
      for (int d = 0; d < DEEP; ++d) w[d].load(wr, k0 + d * a.split * 256, a.K, sw);
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int k = k0 + d * a.split * 256;
        if (!VEC && k - lane * 8 >= a.K) break;
        Piece<VEC> x[T];
#pragma unroll
        for (int t = 0; t < T; ++t) x[t].load(a.x + t * a.ldx, k, a.K, sx);
        float wv[8];
        w[d].take(wr, k, a.K, wv);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          float xv[8];
          x[t].take(a.x + t * a.ldx, k, a.K, xv);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[t] += wv[e] * xv[e];
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
  if (lane == 0)
#pragma unroll
    for (int t = 0; t < T; ++t) s_part[warp][t] = acc[t];
  __syncthreads();
  // one thread per (token, row)
  const int t = threadIdx.x / rows, r = threadIdx.x % rows;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * rows + r;
  if (t >= T || g >= a.N) return;
  float z = 0.f;
  for (int p = 0; p < a.split; ++p) z += s_part[r * a.split + p][t];
  if (a.bias) z += a.bias[g];
  if (a.pre) static_cast<OUT*>(a.pre)[static_cast<int64_t>(t) * a.N + g] = from_f32<OUT>(z);
  float y = act_any(z, a.act);
  if (a.residual) y += to_f32(static_cast<const OUT*>(a.residual)[t * a.ldr + g]);
  static_cast<OUT*>(a.C)[t * a.ldc + g] = from_f32<OUT>(y);
}

template <int T, typename OUT>
cudaError_t launch_typed(const LinearGemm& g, cudaStream_t s) {
  Args a{};
  a.x = static_cast<const __nv_bfloat16*>(g.A);
  a.W = static_cast<const __nv_bfloat16*>(g.B);
  a.ldx = g.lda;
  a.ldw = g.ldb;
  a.ldr = g.ldr;
  a.ldc = g.ldc;
  a.N = g.N;
  a.K = g.K;
  a.act = g.act;
  a.bias = g.bias;
  a.residual = g.residual;
  a.pre = g.pre;
  a.C = g.C;
  // share rows between warps until every SM has its 32, as long as each has a full step
  a.split = 1;
  while (a.split < WARPS && static_cast<int64_t>(g.N) * a.split < static_cast<int64_t>(device_sm_count()) * 32 &&
         g.K >= 256 * DEEP * a.split)
    a.split *= 2;
  const bool vec = ((reinterpret_cast<uintptr_t>(g.A) | reinterpret_cast<uintptr_t>(g.B)) & 15u) == 0 &&
                   g.K % 8 == 0 && g.ldb % 8 == 0 && (T == 1 || g.lda % 8 == 0);
  const int rows = WARPS / a.split;
  const int64_t grid = (static_cast<int64_t>(g.N) + rows - 1) / rows;
  return vec ? launch_overlapped(linear_vec_kernel<T, true, OUT>, grid, 32 * WARPS, 0, s, 0, a)
             : launch_overlapped(linear_vec_kernel<T, false, OUT>, grid, 32 * WARPS, 0, s, 0, a);
}

template <int T>
cudaError_t launch_tokens(const LinearGemm& g, cudaStream_t s) {
  return g.out_dtype == MOE_F32 ? launch_typed<T, float>(g, s) : launch_typed<T, __nv_bfloat16>(g, s);
}

}  // namespace

cudaError_t launch_linear_vec(const LinearGemm& g, cudaStream_t s) {
  switch (g.M) {
    case 1: return launch_tokens<1>(g, s);
    case 2: return launch_tokens<2>(g, s);
    case 3: return launch_tokens<3>(g, s);
    case 4: return launch_tokens<4>(g, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace moe
