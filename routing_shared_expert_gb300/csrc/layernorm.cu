// Normalisation of rows, LAYER or RMS, with the residual add in front of it, and its gradients.
//
//   h = x + r,  mean = sum h / d,  rstd = (sum (h - mean)^2 / d + eps)^(-1/2),  y = (h - mean) rstd w + b
//   xhat = (h - mean) rstd,  g = dy w,
//   dx = rstd (g - sum g / d - xhat sum (g xhat) / d) + dsum,  dw = sum_t dy xhat,  db = sum_t dy
// (RMS: mean = 0, no sum g).  The variance is taken from deviations, never as E h^2 - mean^2.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "row_reduce.cuh"

namespace moe {
namespace {

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
};

__device__ __forceinline__ float load_param(const void* p, int32_t dtype, int32_t c, float none) {
  if (!p) return none;
  return dtype == MOE_F32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const __nv_bfloat16*>(p)[c]);
}

// ------------------------------------------------------------------ any layout --
// Any strides, alignment and length: a CTA per row, its threads on neighbouring values, each pass
// over the row a read (from L1 or L2 but for the first).

template <typename X, typename S, typename Y>
__global__ void __launch_bounds__(256) norm_any_kernel(NormArgs a) {
  __shared__ float part[2][32];
  const int64_t t = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + t * a.ldx;
  const S* r = a.r ? static_cast<const S*>(a.r) + t * a.ldr : nullptr;
  S* s = a.s ? static_cast<S*>(a.s) + t * a.lds : nullptr;
  Y* y = static_cast<Y*>(a.y) + t * a.ldy;
  // a value of the row: of the sum as stored, once it is
  auto value = [&](int c) {
    if (s) return to_f32(s[c]);
    const float v = to_f32(x[c]);
    return r ? v + to_f32(r[c]) : v;
  };
  float v[1] = {0.f};
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    if (s) s[c] = from_f32<S>(to_f32(x[c]) + to_f32(r[c]));
    if (!a.rms) v[0] += value(c);
  }
  float mean = 0.f;
  if (!a.rms) {
    block_sum<1>(v, part[0]);
    mean = v[0] / a.d;
  }
  v[0] = 0.f;
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    const float u = value(c) - mean;
    v[0] += u * u;
  }
  block_sum<1>(v, part[1]);
  const float rstd = 1.f / sqrtf(v[0] / a.d + a.eps);
  for (int c = threadIdx.x; c < a.d; c += blockDim.x)
    y[c] = from_f32<Y>((value(c) - mean) * rstd * load_param(a.w, a.w_dtype, c, 1.f) +
                       load_param(a.b, a.w_dtype, c, 0.f));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[t] = mean;
    if (a.rstd) a.rstd[t] = rstd;
  }
}

template <typename H, typename DY, typename S>
__global__ void __launch_bounds__(256) norm_dx_any_kernel(NormArgs a) {
  __shared__ float part[64];
  const int64_t t = blockIdx.x;
  const H* h = static_cast<const H*>(a.x) + t * a.ldx;
  const DY* dy = static_cast<const DY*>(a.y) + t * a.ldy;
  const S* ds = a.r ? static_cast<const S*>(a.r) + t * a.ldr : nullptr;
  S* dx = static_cast<S*>(a.s) + t * a.lds;
  const float mean = a.rms ? 0.f : a.mean[t], rstd = a.rstd[t];
  float v[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    const float g = to_f32(dy[c]) * load_param(a.w, a.w_dtype, c, 1.f);
    v[0] += g;
    v[1] += g * ((to_f32(h[c]) - mean) * rstd);
  }
  block_sum<2>(v, part);
  const float c1 = a.rms ? 0.f : v[0] / a.d, c2 = v[1] / a.d;
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    const float g = to_f32(dy[c]) * load_param(a.w, a.w_dtype, c, 1.f);
    const float z = rstd * (g - c1 - (to_f32(h[c]) - mean) * rstd * c2);
    dx[c] = from_f32<S>(ds ? z + to_f32(ds[c]) : z);
  }
}

// Column sums of a slot's rows (blockIdx.y): 32 columns by 8 rows at a time, joined in order.
template <typename H, typename DY>
__global__ void __launch_bounds__(256) norm_columns_any_kernel(NormArgs a) {
  __shared__ float part[8][2][32];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float w = 0.f, b = 0.f;
  if (c < a.d) {
    const int64_t per = (a.T + a.slots - 1) / a.slots;
    const int64_t t0 = blockIdx.y * per, t1 = min(a.T, t0 + per);
    for (int64_t t = t0 + g; t < t1; t += 8) {
      const float dy = to_f32(static_cast<const DY*>(a.y)[t * a.ldy + c]);
      const float u = to_f32(static_cast<const H*>(a.x)[t * a.ldx + c]) - (a.rms ? 0.f : a.mean[t]);
      w += dy * (u * a.rstd[t]);
      b += dy;
    }
  }
  part[g][0][lane] = w;
  part[g][1][lane] = b;
  __syncthreads();
  if (g < 2 && c < a.d) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][g][lane];
    a.partial[(static_cast<int64_t>(blockIdx.y) * 2 + g) * a.d + c] = v;
  }
}

// The slots' partial sums of dw (blockIdx.y 0) and db (1), in order: each of 8 groups takes a run
// of slots for 32 columns.
__global__ void __launch_bounds__(256) norm_join_kernel(NormArgs a) {
  __shared__ float part[8][32];
  float* out = blockIdx.y == 0 ? a.dw : a.db;
  if (!out) return;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < a.d) {
    const int per = (a.slots + 7) / 8;
    const int s1 = min(a.slots, (g + 1) * per);
    for (int s = g * per; s < s1; ++s) v += a.partial[(static_cast<int64_t>(s) * 2 + blockIdx.y) * a.d + c];
  }
  part[g][lane] = v;
  __syncthreads();
  if (g == 0 && c < a.d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += part[i][lane];
    out[c] = t;
  }
}

// ---------------------------------------------------------------------- launch --

template <typename X, typename S, typename Y>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t s) {
  norm_any_kernel<X, S, Y><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename S, typename Y>
cudaError_t launch_backward(const NormArgs& a, cudaStream_t s) {
  // the column sums first: dx may overwrite h or dy
  const unsigned cols = static_cast<unsigned>((a.d + 31) / 32);
  if (a.dw || a.db) {
    norm_columns_any_kernel<X, Y><<<dim3(cols, static_cast<unsigned>(a.slots)), 256, 0, s>>>(a);
    norm_join_kernel<<<dim3(cols, 2), 256, 0, s>>>(a);
  }
  if (a.s) norm_dx_any_kernel<X, Y, S><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool BWD, typename X, typename S>
cudaError_t launch_y(const NormArgs& a, int32_t y, cudaStream_t s) {
  if (BWD) return y == MOE_F32 ? launch_backward<X, S, float>(a, s) : launch_backward<X, S, __nv_bfloat16>(a, s);
  return y == MOE_F32 ? launch_forward<X, S, float>(a, s) : launch_forward<X, S, __nv_bfloat16>(a, s);
}
template <bool BWD, typename X>
cudaError_t launch_s(const NormArgs& a, int32_t st, int32_t y, cudaStream_t s) {
  return st == MOE_F32 ? launch_y<BWD, X, float>(a, y, s) : launch_y<BWD, X, __nv_bfloat16>(a, y, s);
}
template <bool BWD>
cudaError_t launch_norm(const NormArgs& a, const moe_layernorm_config& c, cudaStream_t s) {
  return c.x_dtype == MOE_F32 ? launch_s<BWD, float>(a, c.stream_dtype, c.y_dtype, s)
                              : launch_s<BWD, __nv_bfloat16>(a, c.stream_dtype, c.y_dtype, s);
}

// ---------------------------------------------------------------------- checks --

constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxElements = int64_t{1} << 40;

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool elem_aligned(const void* p, int32_t t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == MOE_F32 ? 3u : 1u)) == 0;
}

// Rows of partial column sums: one per CTA of a launch that fills the GPU, fewer where rows are so
// long that the partial sums would be more than the operands.
int32_t norm_slots(int64_t T, int32_t d) {
  const int64_t most = std::min<int64_t>(608, std::max<int64_t>(16, (int64_t{1} << 24) / d));
  return static_cast<int32_t>(std::max<int64_t>(1, std::min(T, most)));
}
size_t norm_workspace(int64_t T, int32_t d) {
  return 256 + static_cast<size_t>(norm_slots(T, d)) * 2 * static_cast<size_t>(d) * 4;
}

// Fills the strides; NULL operands have none to check.
moe_status check_norm(const moe_layernorm_config* c, bool r, bool s, NormArgs& a) {
  if (!c || c->T < 0 || c->T > kMaxRows || c->d < 1 || c->d > kMaxWidth) return MOE_ERR_INVALID_ARG;
  if (c->kind != MOE_LAYERNORM_LAYER && c->kind != MOE_LAYERNORM_RMS) return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(c->x_dtype) || !dtype_ok(c->stream_dtype) || !dtype_ok(c->y_dtype) || !dtype_ok(c->w_dtype))
    return MOE_ERR_INVALID_ARG;
  const int64_t given[4] = {c->ldx, r ? c->ldr : 0, s ? c->lds : 0, c->ldy};
  int64_t* out[4] = {&a.ldx, &a.ldr, &a.lds, &a.ldy};
  for (int i = 0; i < 4; ++i) {
    const int64_t ld = c->T > 1 && given[i] ? given[i] : c->d;
    if (ld < c->d) return MOE_ERR_INVALID_ARG;
    if (c->T > 0 && ld > kMaxElements / c->T) return MOE_ERR_UNSUPPORTED;
    *out[i] = ld;
  }
  a.T = c->T;
  a.d = c->d;
  a.eps = c->eps;
  a.rms = c->kind == MOE_LAYERNORM_RMS;
  a.w_dtype = c->w_dtype;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_layernorm_forward(const moe_layernorm_config* cfg, const void* x,
                                 const void* residual, const void* weight, const void* bias,
                                 void* sum, void* y, float* mean, float* rstd, cudaStream_t stream) {
  using namespace moe;
  NormArgs a{};
  const moe_status st = check_norm(cfg, residual, sum, a);
  if (st != MOE_OK) return st;
  if ((sum && !residual) || (mean && a.rms)) return MOE_ERR_INVALID_ARG;
  if (a.T == 0) return MOE_OK;
  if (!x || !y) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, cfg->x_dtype) || !elem_aligned(residual, cfg->stream_dtype) ||
      !elem_aligned(sum, cfg->stream_dtype) || !elem_aligned(y, cfg->y_dtype) ||
      !elem_aligned(weight, cfg->w_dtype) || !elem_aligned(bias, cfg->w_dtype) ||
      !elem_aligned(mean, MOE_F32) || !elem_aligned(rstd, MOE_F32))
    return MOE_ERR_MISALIGNED;
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.b = bias;
  a.s = sum;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return launch_norm<false>(a, *cfg, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_layernorm_workspace_size(int64_t T, int32_t d, size_t* bytes) {
  using namespace moe;
  if (!bytes || T < 0 || T > kMaxRows || d < 1 || d > kMaxWidth) return MOE_ERR_INVALID_ARG;
  *bytes = norm_workspace(T, d);
  return MOE_OK;
}

moe_status moe_layernorm_backward(const moe_layernorm_config* cfg, const void* h,
                                  const void* weight, const float* mean, const float* rstd,
                                  const void* dy, const void* dsum, void* dx, float* dweight,
                                  float* dbias, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  using namespace moe;
  NormArgs a{};
  const moe_status st = check_norm(cfg, dsum, dx, a);
  if (st != MOE_OK) return st;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (a.T > 0 && (!h || !dy || !rstd || (!mean && !a.rms))) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(h, cfg->x_dtype) || !elem_aligned(dsum, cfg->stream_dtype) ||
      !elem_aligned(dx, cfg->stream_dtype) || !elem_aligned(dy, cfg->y_dtype) ||
      !elem_aligned(weight, cfg->w_dtype) || !elem_aligned(mean, MOE_F32) || !elem_aligned(rstd, MOE_F32) ||
      !elem_aligned(dweight, MOE_F32) || !elem_aligned(dbias, MOE_F32) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MOE_ERR_MISALIGNED;
  if (workspace_bytes < norm_workspace(a.T, a.d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a.T == 0) {
    const size_t bytes = static_cast<size_t>(a.d) * 4;
    if (dweight && cudaMemsetAsync(dweight, 0, bytes, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, bytes, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  a.x = h;
  a.r = dsum;
  a.w = weight;
  a.s = dx;
  a.y = const_cast<void*>(dy);
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dw = dweight;
  a.db = dbias;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  a.slots = norm_slots(a.T, a.d);
  return launch_norm<true>(a, *cfg, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
