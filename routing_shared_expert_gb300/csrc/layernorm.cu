// Normalisation of rows, forward; the checks and entry points of both passes.
#include "layernorm.cuh"

namespace moe {
namespace {

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

template <typename X, typename S, typename Y, int E, bool SPLIT, bool ENDS>
__global__ void __launch_bounds__(E == 32 ? 512 : 1024) norm_vec_kernel(NormArgs a) {
  constexpr int G = kGroup<X, S, Y>, P = E / G, N = G / 2;
  extern __shared__ float4 smem[];
  __shared__ float part[SPLIT ? 1 : kMaxTeams * 2 * 32];
  launch_dependents();
  const Seat<G, P, SPLIT> at(a, phase_of<G>(static_cast<const X*>(a.x) + blockIdx.x * a.ldx));
  const int d = a.d;
  const bool add = a.r != nullptr;
  float* w = reinterpret_cast<float*>(smem);
  float* b = w + (a.w ? G * at.groups : 0);
  Feed<X, G, P, SPLIT, ENDS> x(a.x, a.ldx, at);
  Feed<S, G, P, SPLIT, ENDS> r(a.r, a.ldr, at);
  Sink<S, G, P, SPLIT, ENDS> sum(a.s, a.lds, at);
  Sink<Y, G, P, SPLIT, ENDS> y(a.y, a.ldy, at);
  // the ring: each thread's groups of x, then those of r
  char* const base = reinterpret_cast<char*>(b + (a.b ? G * at.groups : 0));
  char* const ring = base + threadIdx.x * static_cast<uint32_t>(G * sizeof(X));
  const uint32_t at_r = P * x.stride + threadIdx.x * static_cast<uint32_t>(G * sizeof(S)) - threadIdx.x * static_cast<uint32_t>(G * sizeof(X));
  const uint32_t stage_bytes = P * x.stride + (add ? P * r.stride : 0);
  char* const ring_end = ring + a.stages * stage_bytes;
  const int T = static_cast<int>(a.T);
  int ahead = at.row;
  auto fetch = [&](char* to) {
    if (ahead < T) {
      x.copy(to, at, ahead, T);
      if (add) r.copy(to + at_r, at, ahead, T);
    }
    ahead += at.step;
    cp_async_commit();
  };
  wait_for_previous();
  for (char* to = ring; to != ring_end; to += stage_bytes) {
    if (!at.all) {      // groups past the row are never copied
      x.clear(to);
      if (add) r.clear(to + at_r);
    }
    fetch(to);
  }
  if (a.w) stage_param<G>(w, a.w, a.w_dtype, at.groups, at.phase, d);
  if (a.b) stage_param<G>(b, a.b, a.w_dtype, at.groups, at.phase, d);
  __syncthreads();
  const float inv_d = 1.f / d;
  int turn = 0;
  int row = at.row;
  char* from = ring;
  for (int it = 0; it < at.turns; ++it, row += at.step) {
    const bool live = !SPLIT || row < T;
    wait_stage(a.stages);
    if (!live) {
      x.clear(from);
      if (add) r.clear(from + at_r);
    }
    float2 h[P][N];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      x.read(from, k, at, h[k]);
      if (add) {
        float2 v[N];
        r.read(from + at_r, k, at, v);
#pragma unroll
        for (int j = 0; j < N; ++j) h[k][j] = add2(h[k][j], v[j]);
        if (a.s) {
          if (live) sum.store(k, at, h[k]);
          round_to<S>(h[k]);     // normalised is the sum as stored
        }
      }
    }
    fetch(from);
    from += stage_bytes;
    if (from == ring_end) from = ring;
    sum.row += sum.step;
    float v[1];
    float mean = 0.f;
    if (!a.rms) {
      float2 total = both(0.f);
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) total = add2(total, h[k][j]);
      v[0] = total.x + total.y;
      row_sum<SPLIT, 1, 32>(v, part, turn, at.lanes, at.lane, at.team);
      mean = v[0] * inv_d;
#pragma unroll
      for (int k = 0; k < P; ++k) {
#pragma unroll
        for (int j = 0; j < N; ++j) h[k][j] = add2(h[k][j], both(ENDS || at.whole[k] ? -mean : 0.f));
        if (ENDS && !at.whole[k]) {
          asm volatile("");
          keep(h[k], at.mask[k]);
        }
      }
    }
    float2 sq = both(0.f);
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
      for (int j = 0; j < N; ++j) sq = fma2(h[k][j], h[k][j], sq);
    v[0] = sq.x + sq.y;
    row_sum<SPLIT, 1, 32>(v, part, turn, at.lanes, at.lane, at.team);
    const float rstd = rsqrtf(v[0] * inv_d + a.eps);
    if (!live) continue;      // its last turn
    if (at.lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float2 u[N];
#pragma unroll
      for (int j = 0; j < N; ++j) h[k][j] = mul2(h[k][j], both(rstd));
      if (a.w) {
        param_group(w, at.groups, k * at.lanes + at.lane, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[k][j] = mul2(h[k][j], u[j]);
      }
      if (a.b) {
        param_group(b, at.groups, k * at.lanes + at.lane, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[k][j] = add2(h[k][j], u[j]);
      }
      y.store(k, at, h[k]);
    }
    y.row += y.step;
  }
}

// ---------------------------------------------------------------------- launch --

template <typename X, typename S, typename Y, int E, bool SPLIT>
cudaError_t launch_vec(const NormArgs& a, const Plan& p, cudaStream_t s) {
  const auto f = p.ends ? norm_vec_kernel<X, S, Y, E, SPLIT, true> : norm_vec_kernel<X, S, Y, E, SPLIT, false>;
  const cudaError_t e = allow_smem(f, p.smem);
  if (e != cudaSuccess) return e;
  return launch_over(f, dim3(p.grid), p.threads, p.smem, s, a);
}

template <typename X, typename S, typename Y>
cudaError_t launch_forward(NormArgs a, cudaStream_t s) {
  const Plan p = make_plan<X, S, Y>(a, sizeof(X) + (a.r ? sizeof(S) : 0), (a.w != nullptr) + (a.b != nullptr),
                                    int64_t{1} << 30, 1024, 32, 1025);
  a.lanes = p.lanes;
  a.stages = p.stages;
  if (p.elements == 8) return launch_vec<X, S, Y, 8, true>(a, p, s);
  if (p.elements == 16) return p.split ? launch_vec<X, S, Y, 16, true>(a, p, s) : launch_vec<X, S, Y, 16, false>(a, p, s);
  if (p.elements == 32 && p.split) return launch_vec<X, S, Y, 32, true>(a, p, s);
  norm_any_kernel<X, S, Y><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename S>
cudaError_t launch_y(const NormArgs& a, int32_t y, cudaStream_t s) {
  return y == MOE_F32 ? launch_forward<X, S, float>(a, s) : launch_forward<X, S, __nv_bfloat16>(a, s);
}
template <typename X>
cudaError_t launch_s(const NormArgs& a, int32_t st, int32_t y, cudaStream_t s) {
  return st == MOE_F32 ? launch_y<X, float>(a, y, s) : launch_y<X, __nv_bfloat16>(a, y, s);
}
cudaError_t launch_forward_any_type(const NormArgs& a, const moe_layernorm_config& c, cudaStream_t s) {
  const int32_t stream = a.r ? c.stream_dtype : c.x_dtype;    // without a residual: the form of x alone
  return c.x_dtype == MOE_F32 ? launch_s<float>(a, stream, c.y_dtype, s)
                              : launch_s<__nv_bfloat16>(a, stream, c.y_dtype, s);
}

cudaError_t launch_backward_any_type(const NormArgs& a, const moe_layernorm_config& c, cudaStream_t s) {
  const int32_t stream = a.s ? c.stream_dtype : c.x_dtype;    // without dx: the form of h and dy alone
  if (c.x_dtype == MOE_F32)
    return c.y_dtype == MOE_F32 ? launch_layernorm_grad<float, float>(a, stream, s)
                                : launch_layernorm_grad<float, __nv_bfloat16>(a, stream, s);
  return c.y_dtype == MOE_F32 ? launch_layernorm_grad<__nv_bfloat16, float>(a, stream, s)
                              : launch_layernorm_grad<__nv_bfloat16, __nv_bfloat16>(a, stream, s);
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
// long that the partial sums would be more than the operands, never fewer than the eight CTAs that
// rows of every phase take.
int32_t norm_slots(int64_t T, int32_t d) {
  const int64_t most = std::min<int64_t>(608, std::max<int64_t>(16, (int64_t{1} << 24) / d));
  return static_cast<int32_t>(std::max<int64_t>(8, std::min(T, most)));
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
  return launch_forward_any_type(a, *cfg, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  return launch_backward_any_type(a, *cfg, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
