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

// The words of N consecutive groups of four elements from group q on.  Split products (a low and
// a high multiply) measured ahead of wide ones (75 against 87 us for 8192 x 7168), and the calls of
// one thread share the key's additions.
template <int N>
__device__ __forceinline__ void philox4x32(const uint64_t* rng, uint64_t q, uint4 (&c)[N]) {
  const uint64_t seed = __ldg(rng), offset = __ldg(rng + 1);
  uint2 k = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
#pragma unroll
  for (int g = 0; g < N; ++g)
    c[g] = make_uint4(static_cast<uint32_t>(q + g), static_cast<uint32_t>((q + g) >> 32),
                      static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32));
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int g = 0; g < N; ++g) {
      const uint32_t lo0 = c[g].x * 0xD2511F53u, hi0 = __umulhi(c[g].x, 0xD2511F53u);
      const uint32_t lo1 = c[g].z * 0xCD9E8D57u, hi1 = __umulhi(c[g].z, 0xCD9E8D57u);
      c[g] = make_uint4(hi1 ^ c[g].y ^ k.x, lo1, hi0 ^ c[g].w ^ k.y, lo0);
    }
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
}

// Eight consecutive values, from and to memory aligned to their size.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// G groups of eight elements per thread, each one access of each operand, the generator between
// the loads and the stores.  Dense operands are one row of n elements, whatever their shape;
// strided ones have rows of a multiple of eight.
// Bound by memory for large operands: 8192 x 7168, fp32 + bf16 -> bf16, in 66 to 69 us (7.1 to 6.8
// TB/s, by the GB300), 16383 x 2047 bf16 -> fp32 in 30.4 to 32.8 us.  With one group per thread the generator's integer
// products bind instead (75 and 38 us).
template <typename X, typename R, typename Y, bool RES, int G, bool DENSE>
__global__ void __launch_bounds__(256) dropout_vec_kernel(DropoutArgs a) {
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * (8 * G);
  const int64_t n = a.rows * a.cols;
  if (i0 >= n) return;
  int64_t ox[G], oy[G], orr[G];   // where the groups start
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t i = i0 + 8 * g;
    const int64_t row = DENSE ? 0 : i / a.cols, col = i - row * a.cols;
    ox[g] = row * a.ldx + col;
    oy[g] = row * a.ldy + col;
    orr[g] = row * a.ldr + col;
  }
  const X* x = static_cast<const X*>(a.x);
  const R* r = static_cast<const R*>(a.r);
  Y* y = static_cast<Y*>(a.y);
  if (i0 + 8 * G > n) {   // the last thread's rest, one by one and apart: inside, it costs registers
#pragma unroll 1
    for (int64_t i = i0; i < n; ++i) {
      const int64_t row = DENSE ? 0 : i / a.cols, col = i - row * a.cols;
      uint4 u[1];
      philox4x32<1>(a.rng, static_cast<uint64_t>(i) / 4, u);
      const uint32_t w = i % 4 == 0 ? u[0].x : i % 4 == 1 ? u[0].y : i % 4 == 2 ? u[0].z : u[0].w;
      float z = w >= a.threshold && !a.drop_all ? to_f32(x[row * a.ldx + col]) * a.scale : 0.f;
      if (RES) z += to_f32(r[row * a.ldr + col]);
      y[row * a.ldy + col] = from_f32<Y>(z);
    }
    return;
  }
  float v[G][8], q[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    load8(x + ox[g], v[g]);
    if (RES) load8(r + orr[g], q[g]);
  }
  uint4 c[2 * G];
  philox4x32<2 * G>(a.rng, static_cast<uint64_t>(i0) / 4, c);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t w[8] = {c[2 * g].x,     c[2 * g].y,     c[2 * g].z,     c[2 * g].w,
                           c[2 * g + 1].x, c[2 * g + 1].y, c[2 * g + 1].z, c[2 * g + 1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[g][j] = w[j] >= a.threshold && !a.drop_all ? v[g][j] * a.scale : 0.f;
      if (RES) v[g][j] += q[g][j];
    }
    store8(y + oy[g], v[g]);
  }
}

// Any strides and alignment: a thread per group of four consecutive element numbers.
template <typename X, typename R, typename Y, bool RES>
__global__ void __launch_bounds__(256) dropout_any_kernel(DropoutArgs a) {
  const int64_t n = a.rows * a.cols;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4;
  if (i >= n) return;
  int64_t row = i / a.cols, col = i - row * a.cols;
  float v[4], q[4];
  int64_t at[4];
  const int m = static_cast<int>(min(n - i, int64_t{4}));
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < m) {
      v[j] = to_f32(static_cast<const X*>(a.x)[row * a.ldx + col]);
      if (RES) q[j] = to_f32(static_cast<const R*>(a.r)[row * a.ldr + col]);
      at[j] = row * a.ldy + col;
      if (++col == a.cols) {
        col = 0;
        ++row;
      }
    }
  uint4 u[1];
  philox4x32<1>(a.rng, static_cast<uint64_t>(i) / 4, u);
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < m) {
      float z = w[j] >= a.threshold && !a.drop_all ? v[j] * a.scale : 0.f;
      if (RES) z += q[j];
      static_cast<Y*>(a.y)[at[j]] = from_f32<Y>(z);
    }
}

template <typename E>
bool aligned8(const void* p, int64_t ld) {   // rows start on groups of eight elements
  return (reinterpret_cast<uintptr_t>(p) & (8 * sizeof(E) - 1)) == 0 && ld % 8 == 0;
}

template <typename X, typename R, typename Y, bool RES>
cudaError_t launch_typed(DropoutArgs a, cudaStream_t s) {
  if (a.ldx == a.cols && a.ldy == a.cols && (!RES || a.ldr == a.cols)) {   // dense: one long row
    a.cols *= a.rows;
    a.rows = 1;
    a.ldx = a.ldy = a.ldr = 0;
  }
  const int64_t n = a.rows * a.cols;
  const bool vec = aligned8<X>(a.x, a.ldx) && aligned8<Y>(a.y, a.ldy) && (!RES || aligned8<R>(a.r, a.ldr)) &&
                   (a.rows == 1 || a.cols % 8 == 0);
  // One group per thread while there are threads to spare (1024 x 1024: 3.3 us against 3.5; 256 x 64:
  // 1.8 against 2.3), two where the generator would bind.
  const unsigned one = static_cast<unsigned>((n + 2047) / 2048), two = static_cast<unsigned>((n + 4095) / 4096);
  if (vec && n < (int64_t{1} << 21)) {
    if (a.rows == 1) dropout_vec_kernel<X, R, Y, RES, 1, true><<<one, 256, 0, s>>>(a);
    else dropout_vec_kernel<X, R, Y, RES, 1, false><<<one, 256, 0, s>>>(a);
  } else if (vec) {
    if (a.rows == 1) dropout_vec_kernel<X, R, Y, RES, 2, true><<<two, 256, 0, s>>>(a);
    else dropout_vec_kernel<X, R, Y, RES, 2, false><<<two, 256, 0, s>>>(a);
  }
  else
    dropout_any_kernel<X, R, Y, RES><<<static_cast<unsigned>((n + 1023) / 1024), 256, 0, s>>>(a);
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
  // element numbers and offsets stay within 2^40, launches within 2^30 blocks of 1024 elements
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
