// The router's balance loss with its z-loss, per-expert counts and gradient of the logits
// (Section 10 "Routing, Capacity, and Load Balancing", Eq. 30 and 38, per sequence).
//
// With f_si = C_si / (K V_s) held fixed the gradient of N sum_i f_i P_i is
//   softmax   (N / V) p_i (f_i - f.p),      sigmoid   (N / V) p_i (1 - sigma_i) (f_i - f.p),
// f.p = sum_j f_j p_j.  Both forms of f enter only as a difference against a mean under p, and
// sum p = 1, so f is replaced by d_i = f_i - 1/N = (N C_i - K V) / (N K V), whose numerator is
// an exact integer: a balanced batch gives exactly zero instead of a difference of rounded
// numbers.
//
// Sigmoid scores are taken times exp(-min(max z, 0)), which leaves p unchanged and keeps
// p defined where every sigma underflows.
//
// Three launches: the counts (integer atomics, so any order gives the same result), one pass
// over the logits (a warp per row: scores, gradient, and per-tile sums of p and lse^2), and one
// CTA that adds the tiles in order.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kRows = 64;      // tokens per tile; a tile lies in one sequence
constexpr int kWarps = 8;
constexpr int64_t kMaxSeqExperts = int64_t{1} << 20;

struct BalanceArgs {
  const float* logits;
  const int32_t* topk;
  const uint8_t* mask;
  int64_t T, L, S;
  int32_t N, K;
  float coef_b, coef_z;
  const float* grad_scale;
  bool sigmoid;
  int32_t* counts;       // [S][N]
  int32_t* valid;        // [S]
  float* partial;        // [tiles][N] sums of p
  float* partial_z;      // [tiles] sums of lse^2
  int64_t tiles_per_seq, tiles;
  float* P;              // nullable
  float* loss;           // nullable
  float* dlogits;        // nullable
  int32_t* counts_out;   // nullable
  int32_t* status;
};

__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float wmax(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__global__ void __launch_bounds__(256) balance_count_kernel(BalanceArgs a) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= a.T || (a.mask && a.mask[t] == 0)) return;
  const int64_t s = t / a.L;
  atomicAdd(a.valid + s, 1);
  for (int k = 0; k < a.K; ++k) {
    const int e = a.topk[t * a.K + k];
    if (e >= 0 && e < a.N)
      atomicAdd(a.counts + s * a.N + e, 1);
    else if (e != -1)
      set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  }
}

// d_i = (N C - K V) / (N K V)
__device__ __forceinline__ float centred_fraction(int32_t c, int32_t v, int N, int K) {
  const long long num = static_cast<long long>(N) * c - static_cast<long long>(K) * v;
  return static_cast<float>(num) / (static_cast<float>(N) * static_cast<float>(K) * static_cast<float>(v));
}

__global__ void __launch_bounds__(256) balance_rows_kernel(BalanceArgs a) {
  constexpr int C = kMaxExperts / 32;
  __shared__ float s_p[kWarps][kMaxExperts];
  __shared__ float s_z[kWarps];
  __shared__ float s_d[kMaxExperts];
  __shared__ int s_ne[kWarps];
  __shared__ long long s_v[kWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t seq = blockIdx.x / a.tiles_per_seq;
  const int64_t t0 = seq * a.L + (blockIdx.x % a.tiles_per_seq) * kRows;
  const int64_t t1 = min(min(t0 + kRows, (seq + 1) * a.L), a.T);
  // sequences with a valid token, and valid tokens of the batch
  int ne = 0;
  long long tot = 0;
  for (int64_t s = threadIdx.x; s < a.S; s += blockDim.x) {
    ne += a.valid[s] > 0;
    tot += a.valid[s];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ne += __shfl_xor_sync(0xffffffffu, ne, o);
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
  }
  if (lane == 0) {
    s_ne[warp] = ne;
    s_v[warp] = tot;
  }
  const int32_t v = a.valid[seq];
  for (int i = threadIdx.x; i < a.N; i += blockDim.x)
    s_d[i] = v > 0 ? centred_fraction(a.counts[seq * a.N + i], v, a.N, a.K) : 0.f;
  __syncthreads();
  ne = 0;
  tot = 0;
  for (int w = 0; w < kWarps; ++w) {
    ne += s_ne[w];
    tot += s_v[w];
  }
  const float g = a.grad_scale ? *a.grad_scale : 1.f;
  const float kb = v > 0 ? g * a.coef_b * static_cast<float>(a.N) / (static_cast<float>(ne) * static_cast<float>(v)) : 0.f;
  const float kz = tot > 0 ? g * a.coef_z * 2.f / static_cast<float>(tot) : 0.f;
  float acc[C], accz = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j) acc[j] = 0.f;
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    const bool on = !a.mask || a.mask[t] != 0;
    if (!on) {
      if (a.dlogits)
        for (int i = lane; i < a.N; i += 32) a.dlogits[t * a.N + i] = 0.f;
      continue;
    }
    float z[C], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = lane + 32 * j;
      z[j] = i < a.N ? a.logits[t * a.N + i] : -INFINITY;
      m = fmaxf(m, z[j]);
    }
    m = wmax(m);
    const bool any = m > -INFINITY;
    float e[C], sum = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      e[j] = any ? expf(z[j] - m) : 0.f;
      sum += e[j];
    }
    sum = wsum(sum);
    const float lse = any ? m + logf(sum) : 0.f;
    const float inv = any ? 1.f / sum : 0.f;
    float p[C], slope[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      p[j] = e[j] * inv;
      slope[j] = 1.f;
    }
    if (a.sigmoid) {
      const float shift = fminf(m, 0.f);
      float q[C], qs = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float ez = expf(z[j]);
        q[j] = !any ? 0.f : z[j] > 0.f ? 1.f / (1.f + expf(-z[j])) : expf(z[j] - shift) / (1.f + ez);
        slope[j] = 1.f / (1.f + ez);
        qs += q[j];
      }
      qs = wsum(qs);
#pragma unroll
      for (int j = 0; j < C; ++j) q[j] = any ? q[j] / qs : 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        e[j] = p[j];
        p[j] = q[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) e[j] = p[j];
    }
    float dp = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = lane + 32 * j;
      acc[j] += p[j];
      if (i < a.N) dp += s_d[i] * p[j];
    }
    dp = wsum(dp);
    accz += lse * lse;
    if (a.dlogits) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int i = lane + 32 * j;
        if (i < a.N)
          a.dlogits[t * a.N + i] = kb * p[j] * slope[j] * (s_d[i] - dp) + kz * lse * e[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) s_p[warp][lane + 32 * j] = acc[j];
  if (lane == 0) s_z[warp] = accz;
  __syncthreads();
  for (int i = threadIdx.x; i < a.N; i += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += s_p[w][i];
    a.partial[static_cast<int64_t>(blockIdx.x) * a.N + i] = s;
  }
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += s_z[w];
    a.partial_z[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(1024) balance_final_kernel(BalanceArgs a) {
  __shared__ double s_l[1024], s_z[1024];
  __shared__ int s_ne[1024];
  __shared__ long long s_v[1024];
  const int i = threadIdx.x;
  double l = 0.0, z = 0.0;
  int ne = 0;
  long long tot = 0;
  for (int64_t j = i; j < a.S * a.N; j += blockDim.x) {
    const int64_t s = j / a.N;
    const int e = static_cast<int>(j - s * a.N);
    const int32_t v = a.valid[s];
    const int32_t c = a.counts[j];
    double sum = 0.0;
    for (int64_t t = 0; t < a.tiles_per_seq; ++t) sum += a.partial[(s * a.tiles_per_seq + t) * a.N + e];
    const double P = v > 0 ? sum / v : 0.0;
    if (a.P) a.P[j] = static_cast<float>(P);
    if (a.counts_out) a.counts_out[j] = c;
    if (v > 0) l += static_cast<double>(static_cast<long long>(a.N) * c) / (static_cast<double>(a.K) * v) * P;
  }
  for (int64_t t = i; t < a.tiles; t += blockDim.x) z += a.partial_z[t];
  for (int64_t s = i; s < a.S; s += blockDim.x) {
    ne += a.valid[s] > 0;
    tot += a.valid[s];
  }
  s_l[i] = l;
  s_z[i] = z;
  s_ne[i] = ne;
  s_v[i] = tot;
  __syncthreads();
  for (int st = 512; st > 0; st >>= 1) {
    if (i < st) {
      s_l[i] += s_l[i + st];
      s_z[i] += s_z[i + st];
      s_ne[i] += s_ne[i + st];
      s_v[i] += s_v[i + st];
    }
    __syncthreads();
  }
  if (i == 0 && a.loss) {
    const double lb = s_ne[0] > 0 ? s_l[0] / s_ne[0] : 0.0;
    const double lz = s_v[0] > 0 ? s_z[0] / static_cast<double>(s_v[0]) : 0.0;
    a.loss[0] = static_cast<float>(a.coef_b * lb + a.coef_z * lz);
    a.loss[1] = static_cast<float>(lb);
    a.loss[2] = static_cast<float>(lz);
  }
}

struct BalanceLayout {
  size_t counts, valid, partial, partial_z, total;
  int64_t L, S, tiles_per_seq, tiles;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

BalanceLayout balance_layout(const moe_config& c, int64_t seq_len) {
  BalanceLayout b{};
  b.L = seq_len > 0 && seq_len < c.T ? seq_len : (c.T > 0 ? c.T : 1);
  b.S = (c.T + b.L - 1) / b.L;
  b.tiles_per_seq = (b.L + kRows - 1) / kRows;
  b.tiles = b.S * b.tiles_per_seq;
  size_t o = 256;
  b.counts = o;
  o = up256(o + static_cast<size_t>(b.S) * (c.N + 1) * 4);   // counts, then valid: cleared together
  b.valid = b.counts + static_cast<size_t>(b.S) * c.N * 4;
  b.partial = o;
  o = up256(o + static_cast<size_t>(b.tiles) * c.N * 4);
  b.partial_z = o;
  o = up256(o + static_cast<size_t>(b.tiles) * 4);
  b.total = o;
  return b;
}

moe_status check_balance(const moe_config* c, int64_t seq_len) {
  size_t bytes = 0;
  const moe_status s = moe_workspace_size(c, &bytes);   // the layer's own checks
  if (s != MOE_OK) return s;
  if (seq_len < 0) return MOE_ERR_INVALID_ARG;
  if (balance_layout(*c, seq_len).S * c->N > kMaxSeqExperts) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_balance_loss_workspace_size(const moe_config* cfg, int64_t seq_len, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_balance(cfg, seq_len);
  if (s != MOE_OK) return s;
  *bytes = moe::balance_layout(*cfg, seq_len).total;
  return MOE_OK;
}

moe_status moe_balance_loss(const moe_config* cfg, const float* logits, const int32_t* topk_idx,
                            const uint8_t* token_mask, int64_t seq_len, float coef_balance,
                            float coef_z, const float* grad_scale, int32_t* counts, float* P,
                            float* loss, float* dlogits, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  using namespace moe;
  const moe_status s = check_balance(cfg, seq_len);
  if (s != MOE_OK) return s;
  if (!std::isfinite(coef_balance) || !std::isfinite(coef_z) || !workspace) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MOE_ERR_MISALIGNED;
  const void* ptrs[] = {logits, topk_idx, grad_scale, counts, P, loss, dlogits};
  for (const void* p : ptrs)
    if (!aligned4(p)) return MOE_ERR_MISALIGNED;
  const BalanceLayout b = balance_layout(*cfg, seq_len);
  if (workspace_bytes < b.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a{};
  a.logits = logits;
  a.topk = topk_idx;
  a.mask = token_mask;
  a.T = cfg->T;
  a.L = b.L;
  a.S = b.S;
  a.N = cfg->N;
  a.K = cfg->K;
  a.coef_b = coef_balance;
  a.coef_z = coef_z;
  a.grad_scale = grad_scale;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.counts = reinterpret_cast<int32_t*>(ws + b.counts);
  a.valid = reinterpret_cast<int32_t*>(ws + b.valid);
  a.partial = reinterpret_cast<float*>(ws + b.partial);
  a.partial_z = reinterpret_cast<float*>(ws + b.partial_z);
  a.tiles_per_seq = b.tiles_per_seq;
  a.tiles = b.tiles;
  a.P = P;
  a.loss = loss;
  a.dlogits = dlogits;
  a.counts_out = counts;
  a.status = static_cast<int32_t*>(workspace);
  if (a.T > 0) {
    if (cudaMemsetAsync(a.counts, 0, static_cast<size_t>(b.S) * (a.N + 1) * 4, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    balance_count_kernel<<<static_cast<unsigned>((a.T + 255) / 256), 256, 0, stream>>>(a);
    balance_rows_kernel<<<static_cast<unsigned>(a.tiles), 256, 0, stream>>>(a);
  }
  balance_final_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
