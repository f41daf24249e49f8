// Gradients of the normalisation of rows.
#include "layernorm.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ any layout --
// As in the forward pass: a CTA per row for dx, and the columns' sums apart.

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

// The backward pass in one reading of the rows; the columns' sums stay in registers over the CTA's rows
// (B: those of db too) and go out once.  Between the two uses of a row its values stay in the ring.
template <typename H, typename S, typename DY, int P, bool SPLIT, bool B>
__global__ void __launch_bounds__(SPLIT ? 256 : 512) norm_grad_kernel(NormArgs a) {
  extern __shared__ float4 smem[];
  __shared__ float part[2][64];
  const int lanes = SPLIT ? a.lanes : blockDim.x, lane = SPLIT ? threadIdx.x & (lanes - 1) : threadIdx.x;
  const int groups = lanes * P, d = a.d;
  int64_t row = SPLIT ? blockIdx.x + static_cast<int64_t>(threadIdx.x / lanes) * gridDim.x : blockIdx.x;
  const int64_t step = SPLIT ? static_cast<int64_t>(256 / lanes) * gridDim.x : gridDim.x;
  const int turns = static_cast<int>((a.T - blockIdx.x + step - 1) / step);
  const int phase = phase_of(static_cast<const H*>(a.x) + blockIdx.x * a.ldx);
  const bool add = a.r && a.s;
  float* w = reinterpret_cast<float*>(smem);
  const uint32_t stride = blockDim.x * 16;
  const uint32_t at_y = P * kPieces<H> * stride, at_s = at_y + P * kPieces<DY> * stride;
  const uint32_t stage_bytes = at_s + (add ? P * kPieces<S> * stride : 0);
  char* ring = reinterpret_cast<char*>(w + 8 * groups) + threadIdx.x * 16;
  const Extent eh = extent_of(a.x, a.T, a.ldx, d, sizeof(H)), ey = extent_of(a.y, a.T, a.ldy, d, sizeof(DY)),
               es = extent_of(a.r, a.T, a.ldr, d, sizeof(S));
  auto fetch = [&](int64_t t, char* to) {
    if (t < a.T) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int e0 = 8 * (k * lanes + lane) - phase;
        copy_group(to + k * kPieces<H> * stride, stride, static_cast<const H*>(a.x) + t * a.ldx, e0, d, eh);
        copy_group(to + at_y + k * kPieces<DY> * stride, stride, static_cast<const DY*>(a.y) + t * a.ldy, e0, d, ey);
        if (add)
          copy_group(to + at_s + k * kPieces<S> * stride, stride, static_cast<const S*>(a.r) + t * a.ldr, e0, d, es);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < a.stages; ++i) fetch(row + i * step, ring + i * stage_bytes);
  if (a.w) stage_param(w, a.w, a.w_dtype, groups, phase, d);
  __syncthreads();
  const float inv_d = 1.f / d;
  int turn = 0, at = 0;
  float acc_w[P][8], acc_b[P][8];
#pragma unroll
  for (int k = 0; k < P; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc_w[k][j] = acc_b[k][j] = 0.f;
  float mean = 0.f, r = 0.f;
  if (row < a.T) {
    r = a.rstd[row];
    if (!a.rms) mean = a.mean[row];
  }
  for (int it = 0; it < turns; ++it, row += step) {
    const bool live = !SPLIT || row < a.T;
    float next_mean = 0.f, next_r = 0.f;
    if (row + step < a.T) {
      next_r = a.rstd[row + step];
      if (!a.rms) next_mean = a.mean[row + step];
    }
    wait_stage(a.stages);
    char* from = ring + at * stage_bytes;
    at = at + 1 == a.stages ? 0 : at + 1;
    // xhat and g of group k
    auto values = [&](int k, float (&xh)[8], float (&dy)[8], float (&g)[8]) {
      const int q = k * lanes + lane, e0 = 8 * q - phase;
      read_group(from + k * kPieces<H> * stride, stride, static_cast<const H*>(nullptr), xh);
      read_group(from + at_y + k * kPieces<DY> * stride, stride, static_cast<const DY*>(nullptr), dy);
      if (!live || !whole_group(e0, d)) {
        clear_outside(xh, e0, live ? d : 0);
        clear_outside(dy, e0, live ? d : 0);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] = (xh[j] - mean) * r;
        g[j] = dy[j];
      }
      if (a.w) {
        float u[8];
        param8(w, groups, q, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= u[j];
      }
    };
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float xh[8], dy[8], g[8];
      values(k, xh, dy, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc_w[k][j] += dy[j] * xh[j];
        if (B) acc_b[k][j] += dy[j];
        v[0] += g[j];
        v[1] += g[j] * xh[j];
      }
    }
    if (a.s) {
      row_sum<SPLIT, 2>(v, part, turn, lanes);
      const float c1 = a.rms ? 0.f : v[0] * inv_d, c2 = v[1] * inv_d;
      if (live) {
        S* dx = static_cast<S*>(a.s) + row * a.lds;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float xh[8], dy[8], g[8];
          values(k, xh, dy, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = r * (g[j] - c1 - xh[j] * c2);
          if (add) {
            float u[8];
            read_group(from + at_s + k * kPieces<S> * stride, stride, static_cast<const S*>(nullptr), u);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] += u[j];
          }
          store_group(dx, 8 * (k * lanes + lane) - phase, d, g);
        }
      }
    }
    fetch(row + a.stages * step, from);
    mean = next_mean;
    r = next_r;
  }
  if (!a.dw && !a.db) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if (!SPLIT) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int e0 = 8 * (k * lanes + lane) - phase;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e0 + j >= 0 && e0 + j < d) {
          out[e0 + j] = acc_w[k][j];
          if (B) out[d + e0 + j] = acc_b[k][j];
        }
    }
    return;
  }
  // a warp's rows by its lanes, then the warps in order
  float* join = w;
  for (int half = 0; half < (B ? 2 : 1); ++half) {
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (half) acc_w[k][j] = acc_b[k][j];
        for (int o = lanes; o < 32; o <<= 1) acc_w[k][j] += __shfl_xor_sync(0xffffffffu, acc_w[k][j], o);
      }
    for (int i = 0; i < 8; ++i) {
      __syncthreads();
      if ((threadIdx.x >> 5) == i && (threadIdx.x & 31) < lanes)
#pragma unroll
        for (int k = 0; k < P; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 8 * (k * lanes + lane) - phase + j;
            if (c >= 0 && c < d) join[c] = i == 0 ? acc_w[k][j] : join[c] + acc_w[k][j];
          }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) out[half * d + c] = join[c];
  }
}

// ---------------------------------------------------------------------- launch --

template <typename X, typename S, typename Y, int P, bool SPLIT>
cudaError_t launch_grad(const NormArgs& a, const Plan& p, cudaStream_t s) {
  const auto f = a.db ? norm_grad_kernel<X, S, Y, P, SPLIT, true> : norm_grad_kernel<X, S, Y, P, SPLIT, false>;
  const cudaError_t e = allow_smem(f, p.smem);
  if (e != cudaSuccess) return e;
  f<<<p.grid, p.threads, p.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename S, typename Y>
cudaError_t launch_backward(NormArgs a, cudaStream_t s) {
  const unsigned cols = static_cast<unsigned>((a.d + 31) / 32);
  const Plan p = make_plan<X, S, Y>(a, kPieces<X> + kPieces<Y> + (a.r && a.s ? kPieces<S> : 0), 1, a.slots, 512);
  a.lanes = p.lanes;
  a.stages = p.stages;
  cudaError_t e = cudaSuccess;
  if (p.groups_per_thread) {
    if (p.groups_per_thread == 1) e = launch_grad<X, S, Y, 1, true>(a, p, s);
    else if (p.groups_per_thread == 2) e = p.split ? launch_grad<X, S, Y, 2, true>(a, p, s) : launch_grad<X, S, Y, 2, false>(a, p, s);
    else e = launch_grad<X, S, Y, 4, false>(a, p, s);
    if (e != cudaSuccess) return e;
    a.slots = static_cast<int32_t>(p.grid);
    if (a.dw || a.db) norm_join_kernel<<<dim3(cols, 2), 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  // the column sums first: dx may overwrite h or dy
  if (a.dw || a.db) {
    norm_columns_any_kernel<X, Y><<<dim3(cols, static_cast<unsigned>(a.slots)), 256, 0, s>>>(a);
    norm_join_kernel<<<dim3(cols, 2), 256, 0, s>>>(a);
  }
  if (a.s) norm_dx_any_kernel<X, Y, S><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename S>
cudaError_t launch_y(const NormArgs& a, int32_t y, cudaStream_t s) {
  return y == MOE_F32 ? launch_backward<X, S, float>(a, s) : launch_backward<X, S, __nv_bfloat16>(a, s);
}
template <typename X>
cudaError_t launch_s(const NormArgs& a, int32_t st, int32_t y, cudaStream_t s) {
  return st == MOE_F32 ? launch_y<X, float>(a, y, s) : launch_y<X, __nv_bfloat16>(a, y, s);
}

}  // namespace

cudaError_t launch_layernorm_backward(const NormArgs& a, const moe_layernorm_config& c, cudaStream_t s) {
  return c.x_dtype == MOE_F32 ? launch_s<float>(a, c.stream_dtype, c.y_dtype, s)
                              : launch_s<__nv_bfloat16>(a, c.stream_dtype, c.y_dtype, s);
}

}  // namespace moe
