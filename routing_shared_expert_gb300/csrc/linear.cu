// Dense projections of the block: y = act(x W^T + b) + r and the gradients dx, dW, db.
//
//   z = x W^T + b,  y = act(z) + r
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_t dz
//
// The three products are one kernel over operand strides: C[m][n] = sum_k A(m, k) B(n, k), a
// 64 x 64 tile per CTA staged through shared memory in steps of 16, fp32 accumulation.
#include <algorithm>

#include "activation.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int TILE = 64;
constexpr int KSTEP = 16;
constexpr int kDbRows = 256;   // rows per partial sum of db

struct ProductArgs {
  const __nv_bfloat16* A;
  const __nv_bfloat16* B;
  int64_t sam, sak, sbn, sbk;   // element strides
  int64_t M, N, K;
  const float* bias;            // [N]
  const void* residual;         // [M][ldr]
  void* pre;                    // [M][N]
  void* C;                      // [M][ldc]
  int64_t ldr, ldc;
  int32_t act;
};

template <typename OUT>
__global__ void __launch_bounds__(256) product_kernel(ProductArgs a) {
  __shared__ float sA[KSTEP][TILE + 1], sB[KSTEP][TILE + 1];
  const int64_t tiles_n = (a.N + TILE - 1) / TILE;
  const int64_t m0 = blockIdx.x / tiles_n * TILE, n0 = blockIdx.x % tiles_n * TILE;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += KSTEP) {
    for (int i = threadIdx.x; i < TILE * KSTEP; i += 256) {
      const int r = i / KSTEP, k = i % KSTEP;
      const bool kin = k0 + k < a.K;
      sA[k][r] = kin && m0 + r < a.M ? to_f32(a.A[(m0 + r) * a.sam + (k0 + k) * a.sak]) : 0.f;
      sB[k][r] = kin && n0 + r < a.N ? to_f32(a.B[(n0 + r) * a.sbn + (k0 + k) * a.sbk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KSTEP; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sA[k][ty * 4 + i] * sB[k][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      const float z = acc[i][j] + (a.bias ? a.bias[n] : 0.f);
      if (a.pre) static_cast<OUT*>(a.pre)[m * a.N + n] = from_f32<OUT>(z);
      float y = act_value(z, a.act);
      if (a.residual) y += to_f32(static_cast<const OUT*>(a.residual)[m * a.ldr + n]);
      static_cast<OUT*>(a.C)[m * a.ldc + n] = from_f32<OUT>(y);
    }
}

// dz rows (bf16) and, per block of kDbRows rows, their column sums.
template <typename OUT>
__global__ void __launch_bounds__(256) dz_kernel(const void* dy, int64_t ldy, const void* pre, int act,
                                                 int64_t T, int64_t n, __nv_bfloat16* dz, float* part) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= n) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kDbRows;
  const int64_t t1 = min(T, t0 + kDbRows);
  float sum = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    float v = to_f32(static_cast<const OUT*>(dy)[t * ldy + col]);
    if (act != MOE_ACT_NONE) v *= act_slope(to_f32(static_cast<const OUT*>(pre)[t * n + col]), act);
    sum += v;
    dz[t * n + col] = from_f32<__nv_bfloat16>(v);
  }
  part[blockIdx.y * n + col] = sum;
}

__global__ void __launch_bounds__(256) db_kernel(const float* part, int64_t blocks, int64_t n, float* db) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= n) return;
  float sum = 0.f;
  for (int64_t b = 0; b < blocks; ++b) sum += part[b * n + col];
  db[col] = sum;
}

cudaError_t launch_product(const ProductArgs& a, int32_t out_dtype, cudaStream_t s) {
  const int64_t tiles = ((a.M + TILE - 1) / TILE) * ((a.N + TILE - 1) / TILE);
  if (tiles == 0) return cudaSuccess;
  if (out_dtype == MOE_F32)
    product_kernel<float><<<static_cast<unsigned>(tiles), 256, 0, s>>>(a);
  else
    product_kernel<__nv_bfloat16><<<static_cast<unsigned>(tiles), 256, 0, s>>>(a);
  return cudaGetLastError();
}

struct LinearLayout {
  size_t dz, db_part, total;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

LinearLayout linear_layout(const moe_linear_config& c) {
  LinearLayout L{};
  size_t o = 256;
  L.dz = o;
  o = up256(o + static_cast<size_t>(c.T) * c.out_features * 2);
  L.db_part = o;
  o = up256(o + static_cast<size_t>((c.T + kDbRows - 1) / kDbRows) * c.out_features * 4);
  L.total = o;
  return L;
}

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool elem_aligned(const void* p, int32_t t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == MOE_F32 ? 3u : 1u)) == 0;
}

moe_status check_linear(const moe_linear_config* c) {
  if (!c || c->T < 0 || c->T > (int64_t{1} << 28)) return MOE_ERR_INVALID_ARG;
  if (c->in_features < 1 || c->out_features < 1 || c->in_features > (1 << 20) || c->out_features > (1 << 20))
    return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(c->dtype) || !dtype_ok(c->out_dtype) || !dtype_ok(c->dx_dtype) || !dtype_ok(c->dw_dtype))
    return MOE_ERR_INVALID_ARG;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if ((c->ldx && c->ldx < c->in_features) || (c->ldw && c->ldw < c->in_features) ||
      (c->ldr && c->ldr < c->out_features) || (c->ldy && c->ldy < c->out_features))
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  // byte offsets within 2^46, and products of tile counts within 64 bits
  const int64_t most = int64_t{1} << 44;
  for (int64_t ld : {c->ldx, c->ldw, c->ldr, c->ldy})
    if (ld < 0 || ld > most / std::max<int64_t>(1, std::max<int64_t>(c->T, c->out_features)))
      return MOE_ERR_INVALID_ARG;
  if (c->T * std::max<int64_t>(c->in_features, c->out_features) > (int64_t{1} << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_linear_ws(const moe_linear_config& c, void* ws, size_t bytes) {
  if (!ws) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_MISALIGNED;
  return bytes < linear_layout(c).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_linear_workspace_size(const moe_linear_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_linear(cfg);
  if (s != MOE_OK) return s;
  *bytes = moe::linear_layout(*cfg).total;
  return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_config* cfg, const void* x, const void* W,
                              const float* bias, const void* residual, void* pre, void* y,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace moe;
  moe_status s = check_linear(cfg);
  if (s != MOE_OK) return s;
  const moe_linear_config& c = *cfg;
  if ((s = check_linear_ws(c, workspace, workspace_bytes)) != MOE_OK) return s;
  if (c.T == 0) return MOE_OK;
  if (!x || !W || !y) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, MOE_BF16) || !elem_aligned(W, MOE_BF16) || !elem_aligned(bias, MOE_F32) ||
      !elem_aligned(residual, c.out_dtype) || !elem_aligned(pre, c.out_dtype) ||
      !elem_aligned(y, c.out_dtype))
    return MOE_ERR_MISALIGNED;
  ProductArgs a{};
  a.A = static_cast<const __nv_bfloat16*>(x);
  a.B = static_cast<const __nv_bfloat16*>(W);
  a.sam = c.ldx ? c.ldx : c.in_features;
  a.sbn = c.ldw ? c.ldw : c.in_features;
  a.sak = a.sbk = 1;
  a.M = c.T;
  a.N = c.out_features;
  a.K = c.in_features;
  a.bias = bias;
  a.residual = residual;
  a.pre = pre;
  a.C = y;
  a.ldr = c.ldr ? c.ldr : c.out_features;
  a.ldc = c.ldy ? c.ldy : c.out_features;
  a.act = c.act;
  return launch_product(a, c.out_dtype, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_linear_backward(const moe_linear_config* cfg, const void* x, const void* W,
                               const void* pre, const void* dy, void* dx, void* dW, float* dbias,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace moe;
  moe_status s = check_linear(cfg);
  if (s != MOE_OK) return s;
  const moe_linear_config& c = *cfg;
  if ((s = check_linear_ws(c, workspace, workspace_bytes)) != MOE_OK) return s;
  if (!elem_aligned(x, MOE_BF16) || !elem_aligned(W, MOE_BF16) || !elem_aligned(pre, c.out_dtype) ||
      !elem_aligned(dy, c.out_dtype) || !elem_aligned(dx, c.dx_dtype) || !elem_aligned(dW, c.dw_dtype) ||
      !elem_aligned(dbias, MOE_F32))
    return MOE_ERR_MISALIGNED;
  if (c.T == 0) {
    const size_t n = static_cast<size_t>(c.out_features);
    if (dW && cudaMemsetAsync(dW, 0, n * c.in_features * (c.dw_dtype == MOE_F32 ? 4 : 2), stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, n * 4, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dy || (c.act != MOE_ACT_NONE && !pre) || (dW && !x) || (dx && !W)) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(c);
  char* ws = static_cast<char*>(workspace);
  __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(ws + L.dz);
  float* part = reinterpret_cast<float*>(ws + L.db_part);
  const int64_t ldy = c.ldy ? c.ldy : c.out_features, blocks = (c.T + kDbRows - 1) / kDbRows;
  const dim3 grid(static_cast<unsigned>((c.out_features + 255) / 256), static_cast<unsigned>(blocks));
  if (c.out_dtype == MOE_F32)
    dz_kernel<float><<<grid, 256, 0, stream>>>(dy, ldy, pre, c.act, c.T, c.out_features, dz, part);
  else
    dz_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(dy, ldy, pre, c.act, c.T, c.out_features, dz, part);
  if (dbias)
    db_kernel<<<grid.x, 256, 0, stream>>>(part, blocks, c.out_features, dbias);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && dx) {
    ProductArgs a{};
    a.A = dz;
    a.sam = c.out_features;
    a.sak = 1;
    a.B = static_cast<const __nv_bfloat16*>(W);
    a.sbn = 1;
    a.sbk = c.ldw ? c.ldw : c.in_features;
    a.M = c.T;
    a.N = c.in_features;
    a.K = c.out_features;
    a.C = dx;
    a.ldc = c.in_features;
    e = launch_product(a, c.dx_dtype, stream);
  }
  if (e == cudaSuccess && dW) {
    ProductArgs a{};
    a.A = dz;
    a.sam = 1;
    a.sak = c.out_features;
    a.B = static_cast<const __nv_bfloat16*>(x);
    a.sbn = 1;
    a.sbk = c.ldx ? c.ldx : c.in_features;
    a.M = c.out_features;
    a.N = c.in_features;
    a.K = c.T;
    a.C = dW;
    a.ldc = c.in_features;
    e = launch_product(a, c.dw_dtype, stream);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
