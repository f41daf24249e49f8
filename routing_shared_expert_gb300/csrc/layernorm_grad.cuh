// Gradients of the normalisation of rows; the kernels of one pair of types of h and dy are compiled by one file each.
#pragma once

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

// The slots' partial sums of dw (blockIdx.y 0) and db (1), in order: each of 32 warps takes a run of
// slots for 32 columns, all its loads on their way at once (152 slots of 2560: about 3 us behind the gradient launch).
__global__ void __launch_bounds__(1024) norm_join_kernel(NormArgs a) {
  __shared__ float part[32][33];
  float* out = blockIdx.y == 0 ? a.dw : a.db;
  wait_for_previous();
  if (!out) return;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int per = (a.slots + 31) / 32, s0 = g * per, s1 = min(a.slots, s0 + per);
  float v = 0.f;
  if (c < a.d) {
    const float* p = a.partial + (static_cast<int64_t>(s0) * 2 + blockIdx.y) * a.d + c;
#pragma unroll 5
    for (int s = s0; s < s1; ++s, p += 2 * static_cast<int64_t>(a.d)) v += *p;
  }
  part[g][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][g]);
  if (lane == 0 && blockIdx.x * 32 + g < a.d) out[blockIdx.x * 32 + g] = v;
}

// The backward pass in one reading of the rows; the columns' sums stay in registers over the CTA's rows
// (B: those of db too) and go out once.  With c = h - mean and p = dy c:
//   dw = sum p rstd,  dx = rstd (g - c1 - c (rstd c2)),  c1 = sum (dy w) / d,  c2 = rstd sum (p w) / d
// (rstd^2 alone is never formed: it may leave fp32's range where the products do not).
// RMS: no mean and no c1, one sum per row instead of two (db of RMS rows runs the other form).  Between its two
// uses a row stays in registers where a thread has 16 elements of it, else in the ring.
// 32768 x 4096 (LAYER, bf16): 128 us with the join, 6.3 TB/s, HBM and the issue slots (0.6 used) near their limits;
// 8192 x 7168 in fp32 with dsum 139 us, 6.8 TB/s, bound by HBM; 8192 x 2560 (RMS, bf16, dsum) 32 us, of which the join
// and the first and last rows are about 6.  Kept apart, the column sums would read h and dy again.
// Far from that: odd widths, where one team is left to an SM (16384 x 4095 155 us, 16384 x 4096 73), and fp32 rows with
// dsum that leave room for one stage (4096 x 8192 118 us, the bytes at the copy rate 79) or none (2048 x 13376, in the
// general form above, 491 us; 2048 x 13312 96).
template <typename H, typename S, typename DY, int E, bool SPLIT, bool ENDS, bool RMS, bool B>
__global__ void __launch_bounds__(RMS && E <= 16 ? 640 : 512) norm_grad_kernel(NormArgs a) {
  constexpr int G = kGroup<H, S, DY>, P = E / G, N = G / 2;
  extern __shared__ float4 smem[];
  __shared__ float part[SPLIT ? 1 : kMaxTeams * 2 * 32];
  static_assert(sizeof(part) <= kStaticSmem, "the launch counts on no more");
  launch_dependents();
  const Seat<G, P, SPLIT> at(a, phase_of<G>(static_cast<const H*>(a.x) + blockIdx.x * a.ldx));
  const int d = a.d;
  const bool add = a.r && a.s;
  float* w = reinterpret_cast<float*>(smem);
  Feed<H, G, P, ENDS> fh(a.x, a.ldx, at);
  Feed<DY, G, P, ENDS> fy(a.y, a.ldy, at);
  Feed<S, G, P, ENDS> fs(a.r, a.ldr, at);
  Sink<S, G, P, ENDS> dx(a.s, a.lds, at);
  // the ring: each thread's groups of h, then those of dy, then those of dsum
  constexpr uint32_t kH = G * sizeof(H), kY = G * sizeof(DY), kS = G * sizeof(S);
  char* const ring = reinterpret_cast<char*>(w + G * at.groups) + threadIdx.x * kH;
  const uint32_t at_y = P * fh.stride + threadIdx.x * kY - threadIdx.x * kH;
  const uint32_t at_s = P * (fh.stride + fy.stride) + threadIdx.x * kS - threadIdx.x * kH;
  const uint32_t stage_bytes = P * (fh.stride + fy.stride + (add ? fs.stride : 0));
  char* const ring_end = ring + a.stages * stage_bytes;
  const int T = static_cast<int>(a.T);
  int ahead = at.row;
  auto fetch = [&](char* to) {
    if (ahead < T) {
      fh.copy(to, at, ahead, T, a.room);
      fy.copy(to + at_y, at, ahead, T, a.room);
      if (add) fs.copy(to + at_s, at, ahead, T, a.room);
    }
    ahead += at.step;
    cp_async_commit();
  };
  wait_for_previous();
  for (char* to = ring; to != ring_end; to += stage_bytes) {
    if (!at.all) {
      fh.clear_unused(to, at);
      fy.clear_unused(to + at_y, at);
      if (add) fs.clear_unused(to + at_s, at);
    }
    fetch(to);
  }
  if (a.w) stage_param<G>(w, a.w, a.w_dtype, at.groups, at.phase, d);
  __syncthreads();
  const float inv_d = 1.f / d;
  int turn = 0;
  float2 acc_w[P][N], acc_b[P][N];
#pragma unroll
  for (int k = 0; k < P; ++k)
#pragma unroll
    for (int j = 0; j < N; ++j) acc_w[k][j] = acc_b[k][j] = both(0.f);
  int row = at.row;
  float mean = 0.f, r = 0.f;
  if (row < T) {
    r = a.rstd[row];
    if (!RMS && !a.rms) mean = a.mean[row];
  }
  char* from = ring;
  for (int it = 0; it < at.turns; ++it, row += at.step) {
    const bool live = !SPLIT || row < T;
    float next_mean = 0.f, next_r = 0.f;
    if (row + at.step < T) {
      next_r = a.rstd[row + at.step];
      if (!RMS && !a.rms) next_mean = a.mean[row + at.step];
    }
    wait_stage(a.stages);
    if (!live) {
      fh.clear(from);
      fy.clear(from + at_y);
    }
    // c and dy of group k
    auto values = [&](int k, float2 (&c)[N], float2 (&dy)[N]) {
      fh.read(from, k, at, c);
      fy.read(from + at_y, k, at, dy);     // with dy = 0 outside the row nothing there counts
      if (!RMS)
#pragma unroll
        for (int j = 0; j < N; ++j) c[j] = add2(c[j], both(-mean));
    };
    constexpr bool KEEP = E <= 16;
    float2 kc[KEEP ? P : 1][N], kg[KEEP ? P : 1][N];
    float2 sg = both(0.f), sgc = both(0.f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float2 (&c)[N] = kc[KEEP ? k : 0];
      float2 (&g)[N] = kg[KEEP ? k : 0];
      values(k, c, g);
      float2 u[N], p[N];
      if (a.w) {
        param_group(w, at.groups, k * at.lanes + at.lane, u);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) u[j] = both(1.f);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        p[j] = mul2(g[j], c[j]);
        acc_w[k][j] = fma2(p[j], both(r), acc_w[k][j]);
        if (B) acc_b[k][j] = add2(acc_b[k][j], g[j]);
        sgc = fma2(p[j], u[j], sgc);
        if (!RMS) sg = fma2(g[j], u[j], sg);
        if (KEEP) g[j] = mul2(g[j], u[j]);
      }
    }
    if (a.s) {
      float v[RMS ? 1 : 2];
      v[0] = sgc.x + sgc.y;
      if (!RMS) v[RMS ? 0 : 1] = sg.x + sg.y;
      row_sum<SPLIT, RMS ? 1 : 2, 16>(v, part, turn, at.lanes, at.lane, at.team);
      if (live) {
        const float2 c1 = both(RMS || a.rms ? 0.f : -(v[RMS ? 0 : 1] * inv_d) * r), c2 = both(-(v[0] * r * inv_d) * r), rr = both(r);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float2 (&c)[N] = kc[KEEP ? k : 0];
          float2 (&g)[N] = kg[KEEP ? k : 0];
          float2 u[N];
          if (!KEEP) {
            values(k, c, g);
            if (a.w) {
              param_group(w, at.groups, k * at.lanes + at.lane, u);
#pragma unroll
              for (int j = 0; j < N; ++j) g[j] = mul2(g[j], u[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < N; ++j) g[j] = fma2(mul2(c[j], c2), rr, RMS ? mul2(g[j], rr) : fma2(g[j], rr, c1));
          if (add) {
            fs.read(from + at_s, k, at, u);
#pragma unroll
            for (int j = 0; j < N; ++j) g[j] = add2(g[j], u[j]);
          }
          dx.store(k, at, g);
        }
      }
      dx.row += dx.step;
    }
    fetch(from);
    from += stage_bytes;
    if (from == ring_end) from = ring;
    mean = next_mean;
    r = next_r;
  }
  if (!a.dw && !a.db) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
  // every team's sums (SPLIT: every warp's, its rows by its lanes first) to where the ring was, added in order
  const int mine = SPLIT ? threadIdx.x >> 5 : at.team, seats = SPLIT ? blockDim.x >> 5 : blockDim.x / at.lanes;
  const int width = G * at.groups;
  float* join = w + width;
  for (int half = 0; half < (B ? 2 : 1); ++half) {
    if (SPLIT)
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float2& v = half ? acc_b[k][j] : acc_w[k][j];
          for (int o = at.lanes; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          }
        }
    __syncthreads();
    if (!SPLIT || (threadIdx.x & 31) < at.lanes)
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float2 lo = half ? acc_b[k][j] : acc_w[k][j], hi = half ? acc_b[k][j + 1] : acc_w[k][j + 1];
          *reinterpret_cast<float4*>(join + mine * width + G * (k * at.lanes + at.lane) + 2 * j) =
              make_float4(lo.x, lo.y, hi.x, hi.y);
        }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
      float v = join[c + at.phase];
      for (int i = 1; i < seats; ++i) v += join[i * width + c + at.phase];
      out[half * d + c] = v;
    }
  }
}

// ---------------------------------------------------------------------- launch --

template <typename X, typename S, typename Y, int E, bool SPLIT, bool ENDS>
cudaError_t launch_grad_b(const NormArgs& a, const Plan& p, cudaStream_t s) {
  const auto f = a.db    ? norm_grad_kernel<X, S, Y, E, SPLIT, ENDS, false, true>
                 : a.rms ? norm_grad_kernel<X, S, Y, E, SPLIT, ENDS, true, false>
                         : norm_grad_kernel<X, S, Y, E, SPLIT, ENDS, false, false>;
  const cudaError_t e = allow_smem(f, p.smem);
  if (e != cudaSuccess) return e;
  return launch_over(f, dim3(p.grid), p.threads, p.smem, s, a);
}
template <typename X, typename S, typename Y, int E, bool SPLIT>
cudaError_t launch_grad(const NormArgs& a, const Plan& p, cudaStream_t s) {
  return p.ends ? launch_grad_b<X, S, Y, E, SPLIT, true>(a, p, s) : launch_grad_b<X, S, Y, E, SPLIT, false>(a, p, s);
}

template <typename X, typename S, typename Y>
cudaError_t launch_backward(NormArgs a, cudaStream_t s) {
  const unsigned cols = static_cast<unsigned>((a.d + 31) / 32);
  // With two sums a row, many long rows go faster with 32 elements a thread (32768 x 4096: 128 us against 142), few ones
  // slower (64 x 4096: 8.6 against 6.3), and rows over groups too (16384 x 4095: 228 against 164); with one sum there is no
  // difference (8192 x 7168).
  const bool rms = a.rms && !a.db;
  const size_t bytes = sizeof(X) + sizeof(Y) + (a.r && a.s ? sizeof(S) : 0);
  Plan p = make_plan<X, S, Y>(a, bytes, 1, a.slots, rms ? 640 : 512, 16, 513);
  if (!rms && !p.ends && p.elements == 16 && p.lanes >= 256 && a.T >= 16 * device_sm_count())
    p = make_plan<X, S, Y>(a, bytes, 1, a.slots, 512, 16, 256);
  a.lanes = p.lanes;
  a.stages = p.stages;
  a.room = room_of(a, true, kGroup<X, S, Y>);
  if (p.elements) {
    cudaError_t e;
    if (p.elements == 8) e = launch_grad<X, S, Y, 8, true>(a, p, s);
    else if (p.elements == 16) e = p.split ? launch_grad<X, S, Y, 16, true>(a, p, s) : launch_grad<X, S, Y, 16, false>(a, p, s);
    else e = launch_grad<X, S, Y, 32, false>(a, p, s);
    if (e != cudaSuccess) return e;
    a.slots = static_cast<int32_t>(p.grid);
    return a.dw || a.db ? launch_over(norm_join_kernel, dim3(cols, 2), 1024, 0, s, a) : cudaSuccess;
  }
  // the column sums first: dx may overwrite h or dy
  if (a.dw || a.db) {
    norm_columns_any_kernel<X, Y><<<dim3(cols, static_cast<unsigned>(a.slots)), 256, 0, s>>>(a);
    const cudaError_t e = launch_over(norm_join_kernel, dim3(cols, 2), 1024, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.s) norm_dx_any_kernel<X, Y, S><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// The gradients of rows h of X with dy of Y, dsum and dx of the given type.
template <typename X, typename Y>
cudaError_t launch_layernorm_grad(const NormArgs& a, int32_t stream_dtype, cudaStream_t s) {
  return stream_dtype == MOE_F32 ? launch_backward<X, float, Y>(a, s) : launch_backward<X, __nv_bfloat16, Y>(a, s);
}

}  // namespace moe
