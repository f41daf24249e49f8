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

// Forward in one reading.  R: rows that a team takes at a time, which then share the parameters' reads, the barriers
// and the loop.  The mean is taken before the deviations, whose squares are summed from registers.
// 8192 x 7168 (fp32 + bf16 stream -> bf16): 88 us, 6.7 TB/s, bound by HBM (the bytes at the copy rate 86.5 us); rows
// of bf16 alone are bound by the instructions of their sums and parameters: 32768 x 4096 with weight and bias 87 us,
// 6.1 TB/s (one row at a time 101 us at 0.72 issue slots used).  Odd widths pay for the rows' ends and for
// pieces across sectors, and leave some of a warp's lanes idle: 16384 x 4095 73 us, 16384 x 4096 50.  One token of 2048: 2.6 us, the latency of one read.
template <typename X, typename S, typename Y, int E, bool SPLIT, bool ENDS, int R>
__global__ void __launch_bounds__(E == 32 || R == 2 ? 512 : 1024) norm_vec_kernel(NormArgs a) {
  constexpr int G = kGroup<X, S, Y>, P = E / G, N = G / 2;
  extern __shared__ float4 smem[];
  __shared__ float part[SPLIT ? 1 : kMaxTeams * 2 * 32 * R];
  static_assert(sizeof(part) <= kStaticSmem, "the launch counts on no more");
  static_assert(R == 1 || G == 8, "groups of four are taken a row at a time");
  launch_dependents();
  const Seat<G, P, SPLIT, R> at(a, phase_of<G>(static_cast<const X*>(a.x) + blockIdx.x * a.ldx));
  const int d = a.d;
  const bool add = a.r != nullptr;
  float* w = reinterpret_cast<float*>(smem);
  float* b = w + (a.w ? G * at.groups : 0);
  Feed<X, G, P, ENDS> x(a.x, a.ldx, at);
  Feed<S, G, P, ENDS> r(a.r, a.ldr, at);
  Sink<S, G, P, ENDS> sum(a.s, a.lds, at);
  Sink<Y, G, P, ENDS> y(a.y, a.ldy, at);
  // the ring: each thread's groups of x, then those of r; the R rows of a turn in one stage
  char* const base = reinterpret_cast<char*>(b + (a.b ? G * at.groups : 0));
  char* const ring = base + threadIdx.x * static_cast<uint32_t>(G * sizeof(X));
  const uint32_t at_r = P * x.stride + threadIdx.x * static_cast<uint32_t>(G * sizeof(S)) - threadIdx.x * static_cast<uint32_t>(G * sizeof(X));
  const uint32_t row_bytes = P * x.stride + (add ? P * r.stride : 0), stage_bytes = R * row_bytes;
  char* const ring_end = ring + a.stages * stage_bytes;
  const int T = static_cast<int>(a.T);
  int ahead = at.row;
  auto fetch = [&](char* to) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (ahead < T) {
        x.copy(to + i * row_bytes, at, ahead, T, a.room);
        if (add) r.copy(to + i * row_bytes + at_r, at, ahead, T, a.room);
      }
      ahead += at.step;
    }
    cp_async_commit();
  };
  wait_for_previous();
  for (char* to = ring; to != ring_end; to += stage_bytes) {
    if (!at.all)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        x.clear_unused(to + i * row_bytes, at);
        if (add) r.clear_unused(to + i * row_bytes + at_r, at);
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
  for (int it = 0; it < at.turns; ++it, row += R * at.step) {
    bool live[R];
    wait_stage(a.stages);
    float2 h[R][P][N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      live[i] = (!SPLIT && i == 0) || row + i * at.step < T;
      char* const here = from + i * row_bytes;
      if (!live[i]) {
        x.clear(here);
        if (add) r.clear(here + at_r);
      }
#pragma unroll
      for (int k = 0; k < P; ++k) {
        x.read(here, k, at, h[i][k]);
        if (add) {
          float2 v[N];
          r.read(here + at_r, k, at, v);
#pragma unroll
          for (int j = 0; j < N; ++j) h[i][k][j] = add2(h[i][k][j], v[j]);
          if (a.s) {
            if (live[i]) sum.store(k, at, h[i][k], i * sum.step);
            round_to<S>(h[i][k]);     // normalised is the sum as stored
          }
        }
      }
    }
    fetch(from);
    from += stage_bytes;
    if (from == ring_end) from = ring;
    sum.row += R * sum.step;
    float v[R], mean[R];
#pragma unroll
    for (int i = 0; i < R; ++i) mean[i] = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float2 total = both(0.f);
#pragma unroll
        for (int k = 0; k < P; ++k)
#pragma unroll
          for (int j = 0; j < N; ++j) total = add2(total, h[i][k][j]);
        v[i] = total.x + total.y;
      }
      row_sum<SPLIT, R, 32>(v, part, turn, at.lanes, at.lane, at.team);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mean[i] = v[i] * inv_d;
#pragma unroll
        for (int k = 0; k < P; ++k) {
#pragma unroll
          for (int j = 0; j < N; ++j) h[i][k][j] = add2(h[i][k][j], both(ENDS || at.whole[k] ? -mean[i] : 0.f));
          if (ENDS && !at.whole[k]) {
            asm volatile("");
            keep(h[i][k], at.mask[k]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float2 sq = both(0.f);
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) sq = fma2(h[i][k][j], h[i][k][j], sq);
      v[i] = sq.x + sq.y;
    }
    row_sum<SPLIT, R, 32>(v, part, turn, at.lanes, at.lane, at.team);
    float rstd[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      rstd[i] = rsqrtf(v[i] * inv_d + a.eps);
      if (at.lane == 0 && live[i]) {
        if (a.mean) a.mean[row + i * at.step] = mean[i];
        if (a.rstd) a.rstd[row + i * at.step] = rstd[i];
      }
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (G == 8) {
        // Weight and bias in one rounding whether two rows are taken at a time or one, so that a row's bits do not depend
        // on how many rows there are.  R = 2: both parameters on their way at once (32768 x 4096: 88 us, one after the
        // other 109); R = 1: 64 registers leave room for half a group of each.
        constexpr int M = R == 2 ? N : 2;
#pragma unroll
        for (int part = 0; part < N; part += M) {
          float2 u[M], t[M];
          if (a.w) param_values(w, at.groups, k * at.lanes + at.lane, part, u);
          if (a.b) param_values(b, at.groups, k * at.lanes + at.lane, part, t);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < M; ++j) {
              float2& v = h[i][k][part + j];
              v = mul2(v, both(rstd[i]));
              if (a.w && a.b) v = fma2(v, u[j], t[j]);
              else if (a.w) v = mul2(v, u[j]);
              else if (a.b) v = add2(v, t[j]);
            }
        }
      } else {           // groups of four are taken a row at a time; both parameters at once 8192 x 7168 94 -> 101 us
        float2 u[N];
#pragma unroll
        for (int j = 0; j < N; ++j) h[0][k][j] = mul2(h[0][k][j], both(rstd[0]));
        if (a.w) {
          param_group(w, at.groups, k * at.lanes + at.lane, u);
#pragma unroll
          for (int j = 0; j < N; ++j) h[0][k][j] = mul2(h[0][k][j], u[j]);
        }
        if (a.b) {
          param_group(b, at.groups, k * at.lanes + at.lane, u);
#pragma unroll
          for (int j = 0; j < N; ++j) h[0][k][j] = add2(h[0][k][j], u[j]);
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (live[i]) y.store(k, at, h[i][k], i * y.step);
    }
    y.row += R * y.step;
  }
}

// ---------------------------------------------------------------------- launch --

template <typename X, typename S, typename Y, int E, bool SPLIT, int R = 1>
cudaError_t launch_vec(const NormArgs& a, const Plan& p, cudaStream_t s) {
  auto f = norm_vec_kernel<X, S, Y, E, SPLIT, false, R>;
  if constexpr (R == 1)      // two rows at a time: those that end on groups alone
    if (p.ends) f = norm_vec_kernel<X, S, Y, E, SPLIT, true, R>;
  const cudaError_t e = allow_smem(f, p.smem);
  if (e != cudaSuccess) return e;
  return launch_over(f, dim3(p.grid), p.threads, p.smem, s, a);
}

template <typename X, typename S, typename Y>
cudaError_t launch_forward(NormArgs a, cudaStream_t s) {
  const size_t bytes = sizeof(X) + (a.r ? sizeof(S) : 0);
  const int params = (a.w != nullptr) + (a.b != nullptr);
  Plan p = make_plan<X, S, Y>(a, bytes, params, int64_t{1} << 30, 1024, 32, 1025);
  // Rows of bf16 throughout leave the instructions as the bound: two rows at a time share some, where every team has
  // at least two turns of them.
  constexpr bool kBf16 = kGroup<X, S, Y> == 8;
  const bool two = kBf16 && !p.ends && (p.elements == 32 || (p.elements == 16 && !p.split && p.lanes <= 512)) &&
                   a.T >= 4 * static_cast<int64_t>(p.grid) * (p.threads / p.lanes);
  if (two) p = make_plan<X, S, Y>(a, bytes, params, int64_t{1} << 30, 512, 32, 513, 2);
  a.lanes = p.lanes;
  a.stages = p.stages;
  a.room = room_of(a, false, kGroup<X, S, Y>);
  if (two && p.elements == 16) return launch_vec<X, S, Y, 16, false, kBf16 ? 2 : 1>(a, p, s);
  if (two && p.elements == 32 && p.split) return launch_vec<X, S, Y, 32, true, kBf16 ? 2 : 1>(a, p, s);
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
