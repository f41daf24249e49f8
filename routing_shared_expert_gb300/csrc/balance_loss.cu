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
// With E = exp(z): softmax p = E / sum E, sigma = E / (1 + E), 1 - sigma = 1 / (1 + E), so a row
// needs one exponential (and for sigmoid scores one reciprocal) per element, and its three sums
// (E, sigma, d sigma, whose quotient is d.p) go through one shuffle tree.  That holds where
// every |z| < 40; a warp that meets others takes the forms shifted by the row's maximum, with
// sigmoid scores times exp(-min(max z, 0)), which leaves p unchanged and keeps it defined where
// every sigma underflows.
//
// Two launches.  The first counts: a cluster of up to eight CTAs per 4096 tokens of a sequence
// (or 1/16 of it), a histogram in shared memory each, added over distributed shared memory; no
// global atomics.  The second starts under it (programmatic dependent launch) with its first
// logits.  It reads every logit once: W lanes share a row, eight neighbouring logits each (32-byte
// loads where rows allow it), and writes its gradient; the CTAs keep sums of p and lse^2.  The
// last CTA of each 16 of a sequence adds their sums in order, the last of a sequence's groups
// those, the last sequence the losses, whoever that is: the result does not depend on it.
// Sequences short enough for one CTA (four steps of its warps) take one launch, in which each CTA
// counts its own sequence.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kCountThreads = 512;
constexpr int kCountRows = 4096;    // tokens of a counting cluster, while a sequence has
constexpr int kMaxCounts = 16;      // at most so many
constexpr int kCountCtaRows = 512;  // least tokens of a counting CTA
constexpr int kMinSteps = 4;        // least steps of a row CTA's warps
constexpr int64_t kFusedTokens = 16384;   // most tokens whose mask each CTA of the one launch reads
constexpr size_t kFusedTicket = 64;       // bytes into the workspace header: zero between calls
constexpr int kGroup = 16;          // CTAs of a sequence whose sums are added together
constexpr int64_t kMaxSeqExperts = int64_t{1} << 20;
constexpr float kPlain = 40.f;      // |z| below which exp(z) is used as it is

struct BalanceArgs {
  const float* logits;
  const int32_t* topk;
  const uint8_t* mask;
  int64_t T, L, S;
  int32_t N, K;
  float coef_b, coef_z;
  const float* grad_scale;
  bool sigmoid;
  int32_t load_align;    // bytes the rows of logits and dlogits are aligned to: 32, 16 or 4
  bool fused;            // one launch: a CTA per sequence, which counts it too
  int32_t hists;         // counting clusters per sequence
  int32_t count_ctas;    // CTAs of a counting cluster
  int32_t chunks;        // row CTAs per sequence
  int32_t groups;        // ceil(chunks / kGroup)
  int32_t chunk_rows;
  int32_t* hist;         // [S][hists][N + 1]: counts, then valid tokens
  float* partial;        // [S][chunks][N + 1]: sums of p, then of lse^2
  float* gpartial;       // [S][groups][N + 1]
  float* seq;            // [S][2]: N sum f P, sum of lse^2
  unsigned* tickets;     // [S][groups], [S], 1; zeroed by the counting launch
  unsigned* fused_ticket;
  float* P;              // nullable
  float* loss;           // nullable
  float* dlogits;        // nullable
  int32_t* counts;       // nullable
  int32_t* status;
};

__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(BalanceArgs a) {
  __shared__ int s_hist[kMaxExperts + 1];
  launch_dependents();
  const int ctas = a.count_ctas;
  const int rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / ctas;
  const int64_t seq = cluster / a.hists;
  const int part = static_cast<int>(cluster % a.hists) * ctas + rank, parts = a.hists * ctas;
  for (int i = threadIdx.x; i <= a.N; i += blockDim.x) s_hist[i] = 0;
  // this CTA's share of the tickets of the launch that follows
  const int64_t tickets = a.S * (a.groups + 1) + 1;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < tickets;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    a.tickets[i] = 0;
  __syncthreads();
  const int64_t len = min(a.L, a.T - seq * a.L);
  const int64_t t0 = seq * a.L + len * part / parts, t1 = seq * a.L + len * (part + 1) / parts;
  bool bad = false;
  const uint32_t K = static_cast<uint32_t>(a.K), n = static_cast<uint32_t>(t1 - t0) * K;
  const int32_t* topk = a.topk + t0 * a.K;
  const uint8_t* mask = a.mask ? a.mask + t0 : nullptr;
  if (!mask && threadIdx.x == 0) s_hist[a.N] = static_cast<int>(t1 - t0);
  for (uint32_t base = 0; base < n; base += 8 * kCountThreads) {
    int e[8];
    bool on[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t i = base + u * kCountThreads + threadIdx.x, t = i / K;
      e[u] = i < n ? topk[i] : -1;
      on[u] = i < n && (!mask || mask[t] != 0);
      if (mask && on[u] && i == t * K) atomicAdd(&s_hist[a.N], 1);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (!on[u]) continue;
      if (e[u] >= 0 && e[u] < a.N)
        atomicAdd(&s_hist[e[u]], 1);
      else
        bad |= e[u] != -1;
    }
  }
  if (bad) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  if (ctas > 1) cluster_sync_all(); else __syncthreads();
  for (int i = rank * kCountThreads + threadIdx.x; i <= a.N; i += ctas * kCountThreads) {
    int c = s_hist[i];
    if (ctas > 1) {
      c = 0;
      for (int r = 0; r < ctas; ++r) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(&s_hist[i]), r)) : "memory");
        c += v;
      }
    }
    a.hist[cluster * (a.N + 1) + i] = c;
  }
  if (ctas > 1) cluster_sync_all();   // no CTA leaves while another reads its histogram
}

// d_i = (N C - K V) / (N K V)
__device__ __forceinline__ float centred_fraction(int64_t c, int64_t v, int N, int K) {
  const long long num = static_cast<long long>(N) * c - static_cast<long long>(K) * v;
  return static_cast<float>(num) / (static_cast<float>(N) * static_cast<float>(K) * static_cast<float>(v));
}

// Eight neighbouring values of a row; past N the fill.
__device__ __forceinline__ void load_row8(const float* p, int i, int N, int align, float (&z)[8]) {
  if (align == 32) {   // N is a multiple of 8
    if (i < N) {
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(z[0]), "=f"(z[1]), "=f"(z[2]), "=f"(z[3]), "=f"(z[4]), "=f"(z[5]), "=f"(z[6]), "=f"(z[7])
                   : "l"(p + i)
                   : "memory");
      return;
    }
  } else if (align == 16) {   // of 4
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 u = i + 4 * h < N ? *reinterpret_cast<const float4*>(p + i + 4 * h)
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      z[4 * h] = u.x;
      z[4 * h + 1] = u.y;
      z[4 * h + 2] = u.z;
      z[4 * h + 3] = u.w;
    }
    return;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = i + e < N ? p[i + e] : -INFINITY;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = -INFINITY;
}
__device__ __forceinline__ void store_row8(float* p, int i, int N, int align, const float (&v)[8]) {
  if (align == 32) {
    if (i < N)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i), "f"(v[0]), "f"(v[1]),
                   "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
  } else if (align == 16) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (i + 4 * h < N)
        *reinterpret_cast<float4*>(p + i + 4 * h) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < N) p[i + e] = v[e];
  }
}

// The larger value, or NaN where either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Sums and maxima over the W lanes of a row.
template <int W> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int W> __device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Whether this CTA is the last of `n` at the ticket.  Called by the whole CTA, whose writes come
// before what the last one reads.
__device__ __forceinline__ bool last_of(unsigned* ticket, unsigned n) {
  __shared__ bool s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(ticket, 1u) == n - 1;
  __syncthreads();
  const bool last = s_last;
  if (last) __threadfence();
  __syncthreads();
  return last;
}

template <int W, bool SIG>
__global__ void __launch_bounds__(32 * kWarps, SIG ? 3 : 4) balance_rows_kernel(BalanceArgs a) {
  constexpr int G = 32 / W;                   // rows of a warp step
  __shared__ float s_d[kMaxExperts];
  __shared__ float s_p[kWarps][W * 8 + 1];
  __shared__ long long s_red[kWarps][2];
  __shared__ float s_sum[kWarps];
  __shared__ int s_count[kMaxExperts + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t seq = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  const int64_t s0 = seq * a.L, s1 = min(s0 + a.L, a.T);
  const int64_t t0 = s0 + static_cast<int64_t>(chunk) * a.chunk_rows, t1 = min(t0 + a.chunk_rows, s1);
  const int N1 = a.N + 1;
  const int N = a.N;

  // the first logits on their way before the counts are needed (the count launch writes none)
  const int i0 = (lane % W) * 8;
  constexpr int STEP = kWarps * G;
  float z[8];
  bool on = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.f;
  auto fetch = [&](int64_t t) {   // a masked row keeps what was there
    on = t < t1 && (!a.mask || a.mask[t] != 0);
    if (on) load_row8(a.logits + t * N, i0, N, a.load_align, z);
  };
  int64_t t = t0 + warp * G + lane / W;
  fetch(t);
  wait_for_previous();

  // a count of this sequence: requests of expert i, or (i = N) valid tokens
  auto count = [&](int i) {
    long long c = 0;
    if (a.fused) return static_cast<long long>(s_count[i]);
    for (int h = 0; h < a.hists; ++h) c += a.hist[(seq * a.hists + h) * N1 + i];
    return c;
  };
  if (a.fused) {
    for (int i = threadIdx.x; i < N1; i += blockDim.x) s_count[i] = 0;
    __syncthreads();
    bool bad = false;
    const uint32_t K = static_cast<uint32_t>(a.K), n = static_cast<uint32_t>(s1 - s0) * K;
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
      const uint32_t t = i / K;
      if (a.mask && a.mask[s0 + t] == 0) continue;
      if (i == t * K) atomicAdd(&s_count[N], 1);
      const int e = a.topk[s0 * a.K + i];
      if (e >= 0 && e < N)
        atomicAdd(&s_count[e], 1);
      else
        bad |= e != -1;
    }
    if (bad) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    __syncthreads();
  }
  // valid tokens of the batch, and sequences that have one
  long long V, ne;
  if (a.mask && a.fused && a.S == 1) {
    V = s_count[N];
    ne = V > 0;
  } else if (a.mask) {
    long long v = 0, n = 0;
    for (int64_t s = threadIdx.x; s < a.S; s += blockDim.x) {
      int here = 0;
      if (a.fused)
        for (int64_t u = s * a.L; u < min((s + 1) * a.L, a.T); ++u) here += a.mask[u] != 0;
      else
        for (int h = 0; h < a.hists; ++h) here += a.hist[(s * a.hists + h) * N1 + N];
      v += here;
      n += here > 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) {
      s_red[warp][0] = v;
      s_red[warp][1] = n;
    }
    __syncthreads();
    V = ne = 0;
    for (int w = 0; w < kWarps; ++w) {
      V += s_red[w][0];
      ne += s_red[w][1];
    }
  } else {
    V = a.T;
    ne = a.S;
  }
  // this sequence's counts
  const long long vs = count(N);
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    const long long c = count(i);
    s_d[i] = vs > 0 ? centred_fraction(c, vs, N, a.K) : 0.f;
    if (chunk == 0 && a.counts) a.counts[seq * N + i] = static_cast<int32_t>(c);
  }
  __syncthreads();

  const float g = a.grad_scale ? *a.grad_scale : 1.f;
  const float kb = vs > 0 ? g * a.coef_b * static_cast<float>(N) / (static_cast<float>(ne) * static_cast<float>(vs)) : 0.f;
  const float kz = V > 0 ? g * a.coef_z * 2.f / static_cast<float>(V) : 0.f;
  float d[8], acc[8], accz = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    d[e] = i0 + e < N ? s_d[i0 + e] : 0.f;
    acc[e] = 0.f;
  }
  const bool padded = i0 + 8 > N;   // this lane has columns past N, which hold -infinity
  // whole warps take every step: the shuffles need all lanes
  for (int64_t base = t0 + warp * G; base < t1; base += STEP, t += STEP) {
    const bool here = on, in = t < t1;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = z[e];
    fetch(t + STEP);
    // E and the scores p (each times a factor of the row), their slope 1 - sigma, lse, d.p
    float E[8], p[8], slope[8], lse, inv_e, inv_p, dp;
    float reach = 0.f;
    if (!padded) {
#pragma unroll
      for (int e = 0; e < 8; ++e) reach = fmaxf(reach, fabsf(x[e]));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e < N) reach = fmaxf(reach, fabsf(x[e]));
    }
    // fmaxf drops a NaN: where the rest of the warp's logits are small it stays in its row's sums
    if (__all_sync(0xffffffffu, reach < kPlain)) {
      float se = 0.f, sp = 0.f, sd = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        E[e] = exp_ftz(x[e]);
        se += E[e];
        if (SIG) {
          slope[e] = rcp_ftz(1.f + E[e]);
          p[e] = E[e] * slope[e];
          sp += p[e];
        } else {
          p[e] = E[e];
        }
        sd += d[e] * p[e];
      }
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) {
        se += __shfl_xor_sync(0xffffffffu, se, o);
        sd += __shfl_xor_sync(0xffffffffu, sd, o);
        if (SIG) sp += __shfl_xor_sync(0xffffffffu, sp, o);
      }
      inv_e = rcp_ftz(se);
      lse = logf(se);
      inv_p = SIG ? rcp_ftz(sp) : inv_e;
      dp = sd * inv_p;
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, i0 + e < N ? x[e] : -INFINITY);
      m = row_max<W>(m);
      const bool any = !(m == -INFINITY);     // some logit is not -infinity (m is NaN if one is)
      float se = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        E[e] = any && i0 + e < N ? __expf(x[e] - m) : 0.f;
        se += E[e];
      }
      se = row_sum<W>(se);
      inv_e = any ? 1.f / se : 0.f;
      lse = any ? m + logf(se) : 0.f;
      float sp = 0.f, sd = 0.f;
      const float shift = fminf(m, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (SIG) {
          const float ex = __expf(x[e]);
          slope[e] = 1.f / (1.f + ex);        // 0 where ex overflows
          p[e] = !any || i0 + e >= N ? 0.f
                 : x[e] > 0.f        ? 1.f / (1.f + __expf(-x[e]))
                                     : __expf(x[e] - shift) * slope[e];
        } else {
          p[e] = E[e];
        }
        sp += p[e];
        sd += d[e] * p[e];
      }
      sp = row_sum<W>(sp);
      sd = row_sum<W>(sd);
      inv_p = any ? 1.f / sp : 0.f;
      dp = sd * inv_p;
    }
    if (here) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += p[e] * inv_p;
      if (i0 == 0) accz += lse * lse;
    }
    if (a.dlogits && in) {
      float out[8];
      const float kl = kz * lse * inv_e, kp = kb * inv_p;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float b = (d[e] - dp) * (SIG ? p[e] * slope[e] : p[e]);
        out[e] = here ? b * kp + kl * E[e] : 0.f;
      }
      store_row8(a.dlogits + t * N, i0, N, a.load_align, out);
    }
  }

  // the CTA's sums: rows of a warp by shuffles, then the warps in order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = W; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    if (lane < W) s_p[warp][i0 + e] = acc[e];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) accz += __shfl_xor_sync(0xffffffffu, accz, o);
  if (lane == 0) s_p[warp][W * 8] = accz;
  __syncthreads();
  auto cta_sum = [&](int i) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += s_p[w][i < N ? i : W * 8];
    return v;
  };
  const float* from = nullptr;
  if (!a.fused) {
    float* mine = a.partial + (seq * a.chunks + chunk) * N1;
    for (int i = threadIdx.x; i < N1; i += blockDim.x) mine[i] = cta_sum(i);
    // 16 CTAs of a sequence at a time
    const int group = chunk / kGroup, c0 = group * kGroup, c1 = min(a.chunks, c0 + kGroup);
    if (!last_of(a.tickets + seq * a.groups + group, static_cast<unsigned>(c1 - c0))) return;
    from = a.partial + seq * a.chunks * static_cast<int64_t>(N1);
    if (a.groups > 1) {
      for (int i = threadIdx.x; i < N1; i += blockDim.x) {
        float v = 0.f;
#pragma unroll 16
        for (int c = c0; c < c1; ++c) v += __ldcg(from + static_cast<int64_t>(c) * N1 + i);
        a.gpartial[(seq * a.groups + group) * N1 + i] = v;
      }
      if (!last_of(a.tickets + a.S * a.groups + seq, static_cast<unsigned>(a.groups))) return;
      from = a.gpartial + seq * a.groups * static_cast<int64_t>(N1);
    }
  }
  // the sequence: P and its terms of the loss
  const int rows = a.groups > 1 ? a.groups : a.chunks;
  const float inv_v = vs > 0 ? 1.f / static_cast<float>(vs) : 0.f;
  float l = 0.f;
  for (int i = threadIdx.x; i < N1; i += blockDim.x) {
    float v = 0.f;
    if (a.fused) {
      v = cta_sum(i);
    } else {
#pragma unroll 16
      for (int c = 0; c < rows; ++c) v += __ldcg(from + static_cast<int64_t>(c) * N1 + i);
    }
    if (i == N) {
      a.seq[2 * seq + 1] = v;
    } else {
      const float P = v * inv_v;
      if (a.P) a.P[seq * N + i] = P;
      // N f = N C / (K V)
      l += static_cast<float>(static_cast<long long>(N) * count(i)) * inv_v / static_cast<float>(a.K) * P;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_sum[warp] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    l = 0.f;
    for (int w = 0; w < kWarps; ++w) l += s_sum[w];
    a.seq[2 * seq] = l;
  }
  // the batch
  if (a.S == 1) {
    __threadfence_block();
    __syncthreads();
  } else if (a.fused) {
    if (!last_of(a.fused_ticket, static_cast<unsigned>(a.S))) return;
    if (threadIdx.x == 0) *a.fused_ticket = 0;   // for the next call
  } else if (!last_of(a.tickets + a.S * (a.groups + 1), static_cast<unsigned>(a.S))) {
    return;
  }
  if (warp == 0 && a.loss) {
    double lb = 0.0, lz = 0.0;
    for (int64_t s = lane; s < a.S; s += 32) {
      lb += __ldcg(a.seq + 2 * s);
      lz += __ldcg(a.seq + 2 * s + 1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
      lz += __shfl_xor_sync(0xffffffffu, lz, o);
    }
    if (lane == 0) {
      lb = ne > 0 ? lb / static_cast<double>(ne) : 0.0;
      lz = V > 0 ? lz / static_cast<double>(V) : 0.0;
      a.loss[0] = static_cast<float>(a.coef_b * lb + a.coef_z * lz);
      a.loss[1] = static_cast<float>(lb);
      a.loss[2] = static_cast<float>(lz);
    }
  }
}

template <int W>
cudaError_t launch_rows(const BalanceArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.S * a.chunks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // under the count launch
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.fused ? 0 : 1;
  return a.sigmoid ? cudaLaunchKernelEx(&cfg, balance_rows_kernel<W, true>, a)
                   : cudaLaunchKernelEx(&cfg, balance_rows_kernel<W, false>, a);
}

cudaError_t launch_count(const BalanceArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.S * a.hists * a.count_ctas));
  cfg.blockDim = dim3(kCountThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.count_ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, balance_count_kernel, a);
}

struct BalanceLayout {
  size_t hist, partial, gpartial, seq, tickets, total;
  int64_t L, S;
  bool fused;
  int32_t hists, count_ctas, chunks, groups, chunk_rows;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Row CTAs of the whole launch, about: what is resident at once on the GPU this is written for.
constexpr int64_t kSigmoidCtas = 3 * 152, kSoftmaxCtas = 4 * 152;

BalanceLayout balance_layout(const moe_config& c, int64_t seq_len) {
  BalanceLayout b{};
  b.L = seq_len > 0 && seq_len < c.T ? seq_len : (c.T > 0 ? c.T : 1);
  b.S = (c.T + b.L - 1) / b.L;
  b.hists = static_cast<int32_t>(std::min<int64_t>(kMaxCounts, (b.L + kCountRows - 1) / kCountRows));
  b.count_ctas = 1;
  while (b.count_ctas < 8 && b.L / b.hists > b.count_ctas * kCountCtaRows) b.count_ctas *= 2;
  // as many CTAs as keep the GPU in one round, with enough rows to be worth their sums
  int w = 1;   // lanes of a row
  while (w * 8 < c.N) w *= 2;
  const int64_t least = kMinSteps * kWarps * (32 / w);
  const int64_t ctas = c.score == MOE_SCORE_SIGMOID ? kSigmoidCtas : kSoftmaxCtas;
  const int64_t per_seq = b.S > 0 ? std::max<int64_t>(1, ctas / b.S) : 1;
  const int64_t rows = std::max((b.L + per_seq - 1) / per_seq, least);
  b.fused = b.L <= least && c.T <= kFusedTokens;
  b.chunk_rows = static_cast<int32_t>(rows);
  b.chunks = static_cast<int32_t>((b.L + rows - 1) / rows);
  b.groups = (b.chunks + kGroup - 1) / kGroup;
  const size_t S = static_cast<size_t>(b.S), n1 = static_cast<size_t>(c.N) + 1;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  b.hist = take(S * b.hists * n1 * 4);
  b.partial = take(S * b.chunks * n1 * 4);
  b.gpartial = take(S * b.groups * n1 * 4);
  b.seq = take(S * 8);
  b.tickets = take((S * (b.groups + 1) + 1) * 4);
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
  a.load_align = 4;
  const uintptr_t rows = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits) |
                         (static_cast<uintptr_t>(a.N) * 4);
  if (rows % 32 == 0) a.load_align = 32;
  else if (rows % 16 == 0) a.load_align = 16;
  a.hists = b.hists;
  a.count_ctas = b.count_ctas;
  a.chunks = b.chunks;
  a.groups = b.groups;
  a.chunk_rows = b.chunk_rows;
  a.hist = reinterpret_cast<int32_t*>(ws + b.hist);
  a.partial = reinterpret_cast<float*>(ws + b.partial);
  a.gpartial = reinterpret_cast<float*>(ws + b.gpartial);
  a.seq = reinterpret_cast<float*>(ws + b.seq);
  a.tickets = reinterpret_cast<unsigned*>(ws + b.tickets);
  a.P = P;
  a.loss = loss;
  a.dlogits = dlogits;
  a.counts = counts;
  a.status = static_cast<int32_t*>(workspace);
  if (a.T == 0)
    return loss && cudaMemsetAsync(loss, 0, 12, stream) != cudaSuccess ? MOE_ERR_CUDA : MOE_OK;
  a.fused = b.fused;
  a.fused_ticket = reinterpret_cast<unsigned*>(ws + kFusedTicket);
  if (!a.fused && launch_count(a, stream) != cudaSuccess) return MOE_ERR_CUDA;
  const int w = (a.N + 7) / 8;
  const cudaError_t e = w <= 1    ? launch_rows<1>(a, stream)
                        : w <= 2  ? launch_rows<2>(a, stream)
                        : w <= 4  ? launch_rows<4>(a, stream)
                        : w <= 8  ? launch_rows<8>(a, stream)
                        : w <= 16 ? launch_rows<16>(a, stream)
                                  : launch_rows<32>(a, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
