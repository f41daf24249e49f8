// Residual dropout whose mask is never stored: y = r + keep x / (1 - p), and its backward
// pass dx = keep dy / (1 - p).
//
// The keep decision of element i is word i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, 2011) at counter (i div 4, offset) under key seed: ten rounds of two 32 x 32 -> 64-bit
// products, exclusive-ors and a key that grows by two constants.  Both passes compute the
// words from the counter, so nothing of the mask is read or written.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

struct DropoutArgs {
  const void* x;
  const void* r;
  void* y;
  const uint64_t* rng;
  int64_t rows, cols, ldx, ldr, ldy;
  uint32_t threshold;   // kept when the word is >= threshold
  float scale;          // 1 / (1 - p)
  bool drop_all;        // p rounds to 1: the threshold 2^32 does not fit
};

__device__ __forceinline__ uint4 philox4x32(uint4 c, uint2 k) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint32_t lo0 = c.x * 0xD2511F53u, hi0 = __umulhi(c.x, 0xD2511F53u);
    const uint32_t lo1 = c.z * 0xCD9E8D57u, hi1 = __umulhi(c.z, 0xCD9E8D57u);
    c = make_uint4(hi1 ^ c.y ^ k.x, lo1, hi0 ^ c.w ^ k.y, lo0);
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

// One thread per group of four consecutive elements.
template <typename X, typename R, typename Y, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutArgs a) {
  const int64_t n = a.rows * a.cols;
  const int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (q * 4 >= n) return;
  const uint64_t seed = a.rng[0], offset = a.rng[1];
  const uint4 w = philox4x32(make_uint4(static_cast<uint32_t>(q), static_cast<uint32_t>(q >> 32),
                                        static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)),
                             make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)));
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = q * 4 + j;
    if (i >= n) return;
    const int64_t row = i / a.cols, col = i - row * a.cols;
    const bool keep = words[j] >= a.threshold && !a.drop_all;
    float v = keep ? to_f32(static_cast<const X*>(a.x)[row * a.ldx + col]) * a.scale : 0.f;
    if (RES) v += to_f32(static_cast<const R*>(a.r)[row * a.ldr + col]);
    static_cast<Y*>(a.y)[row * a.ldy + col] = from_f32<Y>(v);
  }
}

template <typename X, typename R, typename Y, bool RES>
cudaError_t launch_typed(const DropoutArgs& a, cudaStream_t s) {
  const int64_t groups = (a.rows * a.cols + 3) / 4;
  dropout_kernel<X, R, Y, RES><<<static_cast<unsigned>((groups + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename Y>
cudaError_t launch_xy(const DropoutArgs& a, int32_t r_dtype, cudaStream_t s) {
  if (!a.r) return launch_typed<X, float, Y, false>(a, s);
  return r_dtype == MOE_F32 ? launch_typed<X, float, Y, true>(a, s)
                            : launch_typed<X, __nv_bfloat16, Y, true>(a, s);
}

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool elem_aligned(const void* p, int32_t t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == MOE_F32 ? 3u : 1u)) == 0;
}

moe_status run_dropout(const moe_dropout_config* c, const void* x, int32_t x_dtype, int64_t ldx,
                       const void* r, const uint64_t* rng, void* y, int32_t y_dtype, int64_t ldy,
                       cudaStream_t s) {
  if (!c || c->rows < 0 || c->cols < 0 || !(c->p >= 0.0 && c->p <= 1.0)) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(c->x_dtype) || !dtype_ok(c->y_dtype) || !dtype_ok(c->residual_dtype))
    return MOE_ERR_INVALID_ARG;
  const int64_t lr = c->ldr ? c->ldr : c->cols, lx = ldx ? ldx : c->cols, ly = ldy ? ldy : c->cols;
  if (lx < c->cols || ly < c->cols || lr < c->cols) return MOE_ERR_INVALID_ARG;
  if (c->rows == 0 || c->cols == 0) return MOE_OK;
  // element numbers and offsets stay within 2^40, launches within 2^31 blocks of 1024 elements
  const int64_t most = int64_t{1} << 40;
  if (c->rows > most || lx > most / c->rows || ly > most / c->rows || (r && lr > most / c->rows))
    return MOE_ERR_UNSUPPORTED;
  if (!x || !y || !rng) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, x_dtype) || !elem_aligned(y, y_dtype) ||
      (r && !elem_aligned(r, c->residual_dtype)) || (reinterpret_cast<uintptr_t>(rng) & 7u) != 0)
    return MOE_ERR_MISALIGNED;
  DropoutArgs a{};
  a.x = x;
  a.r = r;
  a.y = y;
  a.rng = rng;
  a.rows = c->rows;
  a.cols = c->cols;
  a.ldx = lx;
  a.ldr = lr;
  a.ldy = ly;
  const double t = std::floor(c->p * 4294967296.0 + 0.5);
  a.drop_all = t >= 4294967296.0;
  a.threshold = a.drop_all ? 0xffffffffu : static_cast<uint32_t>(t);
  a.scale = c->p < 1.0 ? static_cast<float>(1.0 / (1.0 - c->p)) : 0.f;
  cudaError_t e;
  if (x_dtype == MOE_F32)
    e = y_dtype == MOE_F32 ? launch_xy<float, float>(a, c->residual_dtype, s)
                           : launch_xy<float, __nv_bfloat16>(a, c->residual_dtype, s);
  else
    e = y_dtype == MOE_F32 ? launch_xy<__nv_bfloat16, float>(a, c->residual_dtype, s)
                           : launch_xy<__nv_bfloat16, __nv_bfloat16>(a, c->residual_dtype, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_dropout_add(const moe_dropout_config* cfg, const void* x, const void* residual,
                           const uint64_t* rng_state, void* y, cudaStream_t stream) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  return moe::run_dropout(cfg, x, cfg->x_dtype, cfg->ldx, residual, rng_state, y, cfg->y_dtype,
                          cfg->ldy, stream);
}

moe_status moe_dropout_backward(const moe_dropout_config* cfg, const void* dy,
                                const uint64_t* rng_state, void* dx, cudaStream_t stream) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  return moe::run_dropout(cfg, dy, cfg->y_dtype, cfg->ldy, nullptr, rng_state, dx, cfg->x_dtype,
                          cfg->ldx, stream);
}

}  // extern "C"
