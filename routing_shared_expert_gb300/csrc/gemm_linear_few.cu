// The dense projection for few tokens: y = act(x W^T + b) + r bound by reading W once.
//
// The MMA's rows are 128 output features and its columns NT tokens (tcgen05, M = 128, N = NT,
// one CTA), so a tile streams 128 weight rows and a token costs no more tensor work than it
// needs.  out / 128 tiles are too few to keep 152 SMs reading, so the CTAs of a cluster split
// the depth: each accumulates its range of K in its own TMEM, writes the partial sums to its
// shared memory, and after a cluster barrier each CTA adds the partials of its share of the
// tokens in rank order over distributed shared memory (a fixed order, so every call gives the
// same bits, and no second launch or global scratch).  There a warp takes a token and a lane
// four neighbouring features, several tokens at a time, so that the remote reads, the
// residual's reads and the stores of one group overlap.
//
// For fp32 outputs the sum of a CTA is taken in segments of at most 512 deep (as TMEM allows),
// each in its own TMEM columns, and added in rounded fp32: the tensor core's additions drop
// bits, an error that grows with the length of a sum.
//
// The ring holds one 64-wide K block per stage (16 KB of W, 128 NT bytes of x), about 100 KB, so
// that two CTAs share an SM and one streams while the other starts or ends.  More than 64 tokens
// are tiles of 64 (measured ahead of one wider tile, whose CTAs are too few: 256 tokens of 2048 x
// 2048 in 10.1 us against 10.6 with tiles of 128 and 12.5 with 256).
//
// Every wait is bounded; a wait that runs out records MOE_ERR_TIMEOUT and the CTA waits for
// what it issued before it frees its TMEM.
#include <algorithm>
#include <type_traits>

#include "activation.cuh"
#include "linear.h"

namespace moe {
namespace {

constexpr int FM = 128;                    // features per tile
constexpr int BK = 64;
constexpr int W_BYTES = FM * BK * 2;
constexpr int THREADS = 192;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 100000000ull;

template <int NT> struct Shape {
  static constexpr int X_BYTES = NT * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int STAGES = NT <= 16 ? 6 : NT <= 32 ? 5 : 4;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr size_t SMEM = 1024 + RING_BYTES + 8 * (2 * STAGES + 2) + 32;
  static_assert(SMEM <= 113 * 1024, "two CTAs share an SM");
  // fp32 segments in one CTA's half of the 512 TMEM columns
  static constexpr int MAX_SEGMENTS = 256 / (NT < 32 ? 32 : NT);
  static_assert(NT * FM * 4 <= RING_BYTES, "the partial sums take the ring's place");
};

struct Args {
  int32_t T, N, K;         // tokens, features, depth
  int32_t t_tiles;
  int32_t split;           // CTAs per cluster
  int32_t segments;        // TMEM accumulators of a CTA's depth range
  uint32_t tmem_cols;
  const float* bias;
  const void* residual;
  void* pre;
  void* C;
  int64_t ldr, ldc;
  int32_t* status;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four neighbouring output values of a lane.
template <typename OUT> struct alignas(4 * sizeof(OUT)) Four {
  OUT v[4];
  __device__ Four() {}
  __device__ explicit Four(const float (&z)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = from_f32<OUT>(z[e]);
  }
  using Word = typename std::conditional<sizeof(OUT) == 4, uint4, uint2>::type;
  __device__ void load(const OUT* p, bool vec, int n) {
    if (vec) {
      *reinterpret_cast<Word*>(v) = *reinterpret_cast<const Word*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = e < n ? p[e] : from_f32<OUT>(0.f);
    }
  }
  __device__ void store(OUT* p, bool vec, int n) const {
    if (vec) {
      *reinterpret_cast<Word*>(p) = *reinterpret_cast<const Word*>(v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) p[e] = v[e];
    }
  }
  __device__ void add_to(float (&z)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] += to_f32(v[e]);
  }
};

template <int NT, typename OUT, int ACT>
__global__ void __launch_bounds__(THREADS, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const Args args) {
  using S = Shape<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::RING_BYTES);
  uint64_t* empty = full + S::STAGES;
  uint64_t* tfull = empty + S::STAGES;
  uint64_t* drain = tfull + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* never = const_cast<int*>(abort_flag) + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = args.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint32_t smem_base = smem_u32(smem);
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int f0 = tile / args.t_tiles * FM;            // the token tiles of one weight tile together
  const int t0 = tile % args.t_tiles * NT;
  const int k_blocks = (args.K + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(k_blocks) * rank / split);
  const int kbs = static_cast<int>(static_cast<int64_t>(k_blocks) * (rank + 1) / split) - kb0;

  auto load = [&](int i) {                            // K block kb0 + i into its stage
    const int s = i % S::STAGES;
    const uint32_t at = smem_base + s * S::STAGE_BYTES;
    mbar_arrive_expect_tx(smem_u32(&full[s]), S::STAGE_BYTES);
    tma_load_2d(at, &tmW, (kb0 + i) * BK, f0, smem_u32(&full[s]));
    tma_load_2d(at + W_BYTES, &tmX, (kb0 + i) * BK, t0, smem_u32(&full[s]));
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *never = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
    launch_dependents();
    wait_for_previous();
    for (int i = 0; i < S::STAGES && i < kbs; ++i) load(i);   // before the other warps are ready
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_holder), args.tmem_cols);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  wait_for_previous();
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------------- producer
    if (lane == 0) {
      int i = S::STAGES;
      for (; i < kbs; ++i) {
        const int use = i / S::STAGES;
        if (!mbar_wait_bounded(smem_u32(&empty[i % S::STAGES]), (use & 1) ^ 1, abort_flag, args.status,
                               kWaitLimitNs)) {
          ok = false;
          break;
        }
        load(i);
      }
      if (!ok)   // the blocks issued last, one per stage
        for (int j = max(0, i - S::STAGES); j < i; ++j)
          mbar_wait_bounded(smem_u32(&full[j % S::STAGES]), (j / S::STAGES) & 1, never, nullptr,
                            kDrainLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(FM, NT);
      constexpr int SEG_COLS = NT < 32 ? 32 : NT;
      int seg = 0, seg_end = kbs / args.segments;   // segment g ends at (g + 1) kbs / segments
      bool first = true;
      for (int i = 0; i < kbs; ++i) {
        if (i == seg_end) {
          ++seg;
          seg_end = static_cast<int>(static_cast<int64_t>(kbs) * (seg + 1) / args.segments);
          first = true;
        }
        const int s = i % S::STAGES;
        if (!mbar_wait_bounded(smem_u32(&full[s]), (i / S::STAGES) & 1, abort_flag, args.status,
                               kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = smem_base + s * S::STAGE_BYTES;
#pragma unroll
        for (int j = 0; j < BK / 16; ++j)
          tc_mma_bf16(tmem_base + static_cast<uint32_t>(seg * SEG_COLS), sw128_kmajor_desc(at) + 2 * j,
                      sw128_kmajor_desc(at + W_BYTES) + 2 * j, idesc, (!first || j > 0) ? 1u : 0u);
        first = false;
        tc_commit(smem_u32(&empty[s]));
      }
      if (ok) {
        tc_commit(smem_u32(tfull));
      } else {
        tc_commit(smem_u32(drain));
        mbar_wait_bounded(smem_u32(drain), 0, never, nullptr, kDrainLimitNs);
      }
    }
  } else {
    // ------------------------------------------- partial sums to shared memory
    ok = mbar_wait_bounded(smem_u32(tfull), 0, abort_flag, args.status, kWaitLimitNs);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      constexpr int SEG_COLS = NT < 32 ? 32 : NT;
      constexpr int W = NT < 32 ? NT : 32;
      const int q = warp & 3;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;   // [NT][FM]: the ring is idle
#pragma unroll 1
      for (int c = 0; c < NT && t0 + c < args.T; c += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c, v);
        for (int g = 1; g < args.segments; ++g) {
          uint32_t u[32];
          tmem_ld32(taddr + g * SEG_COLS + c, u);
#pragma unroll
          for (int j = 0; j < W; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
        }
#pragma unroll
        for (int j = 0; j < W; ++j) part[(c + j) * FM] = __uint_as_float(v[j]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1) cluster_sync_all(); else __syncthreads();   // every partial sum is in place
  {
    // ------------------------------------------- join, epilogue, output (all warps)
    const int f = f0 + lane * 4;
    const int tokens = min(NT, args.T - t0);
    float b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = args.bias && f + e < args.N ? args.bias[f + e] : 0.f;
    constexpr int WARPS = THREADS / 32, UNROLL = 4;
    constexpr int VEC = 4 * sizeof(OUT);   // bytes of a lane's four values
    // whole groups of four go as one access where every row's groups are aligned to it
    const bool whole = f + 4 <= args.N;
    const bool vec_y = whole && args.ldc % 4 == 0 && (reinterpret_cast<uintptr_t>(args.C) & (VEC - 1)) == 0;
    const bool vec_r = whole && args.ldr % 4 == 0 && (reinterpret_cast<uintptr_t>(args.residual) & (VEC - 1)) == 0;
    const bool vec_p = whole && args.N % 4 == 0 && (reinterpret_cast<uintptr_t>(args.pre) & (VEC - 1)) == 0;
    // this CTA's tokens are rank, rank + split, ...
    for (int j0 = warp; rank + j0 * split < tokens && f < args.N; j0 += WARPS * UNROLL) {
      float4 p[UNROLL];
      Four<OUT> r[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int j = rank + (j0 + u * WARPS) * split;
        if (j >= tokens) break;
        if (args.residual)
          r[u].load(static_cast<const OUT*>(args.residual) + (t0 + j) * args.ldr + f, vec_r, args.N - f);
        const uint32_t at = smem_base + static_cast<uint32_t>(j * FM + lane * 4) * 4u;
        if (split == 1) {
          p[u] = *reinterpret_cast<const float4*>(smem + (j * FM + lane * 4) * 4);
        } else {
          p[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < split; ++k) {
            const float4 o = ld_cluster_f32x4(mapa_shared(at, k));
            p[u] = make_float4(p[u].x + o.x, p[u].y + o.y, p[u].z + o.z, p[u].w + o.w);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int j = rank + (j0 + u * WARPS) * split;
        if (j >= tokens) break;
        const int64_t t = t0 + j;
        float z[4] = {p[u].x + b[0], p[u].y + b[1], p[u].z + b[2], p[u].w + b[3]};
        if (args.pre) Four<OUT>(z).store(static_cast<OUT*>(args.pre) + t * args.N + f, vec_p, args.N - f);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = act_value<ACT>(z[e]);
        if (args.residual) r[u].add_to(z);
        Four<OUT>(z).store(static_cast<OUT*>(args.C) + t * args.ldc + f, vec_y, args.N - f);
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while another reads its partial sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, args.tmem_cols);
  }
}

template <int NT, typename OUT, int ACT>
cudaError_t launch_typed(const LinearGemm& g, int split, cudaStream_t s) {
  using S = Shape<NT>;
  Args a{};
  a.T = static_cast<int32_t>(g.M);
  a.N = g.N;
  a.K = g.K;
  a.t_tiles = (a.T + NT - 1) / NT;
  a.split = split;
  // segments of at most 512 deep for fp32 outputs, one otherwise
  const int cta_blocks = ((a.K + BK - 1) / BK + split - 1) / split;
  a.segments = sizeof(OUT) == 4 ? std::min(S::MAX_SEGMENTS, std::max(1, (cta_blocks + 7) / 8)) : 1;
  a.segments = std::min(a.segments, std::max(1, (a.K + BK - 1) / BK / split));   // none empty
  a.tmem_cols = 32;
  while (a.tmem_cols < static_cast<uint32_t>(a.segments * (NT < 32 ? 32 : NT))) a.tmem_cols *= 2;
  a.bias = g.bias;
  a.residual = g.residual;
  a.pre = g.pre;
  a.C = g.C;
  a.ldr = g.ldr;
  a.ldc = g.ldc;
  a.status = g.status;
  CUtensorMap mW, mX;
  if (!make_strided_map(&mW, MOE_BF16, g.B, g.K, g.N, g.ldb, BK, FM) ||
      !make_strided_map(&mX, MOE_BF16, g.A, g.K, static_cast<uint64_t>(g.M), g.lda, BK, NT))
    return cudaErrorInvalidValue;
  auto kern = linear_few_kernel<NT, OUT, ACT>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, static_cast<int64_t>((a.N + FM - 1) / FM) * a.t_tiles * split, THREADS, S::SMEM, s, split,
                           mW, mX, a);
}

template <typename OUT, int ACT>
cudaError_t launch_out(const LinearGemm& g, cudaStream_t s) {
  const FewShape f = few_shape(g.M, g.N, g.K, device_sm_count());
  switch (f.tokens) {
    case 16: return launch_typed<16, OUT, ACT>(g, f.split, s);
    case 32: return launch_typed<32, OUT, ACT>(g, f.split, s);
    default: return launch_typed<64, OUT, ACT>(g, f.split, s);
  }
}

template <typename OUT>
cudaError_t launch_act(const LinearGemm& g, cudaStream_t s) {
#define MOE_CALL(ACT) launch_out<OUT, ACT>(g, s)
  MOE_DISPATCH_ACT(g.act, MOE_CALL)
#undef MOE_CALL
}

}  // namespace

FewShape few_shape(int64_t T, int64_t N, int64_t K, int sms) {
  FewShape f;
  f.tokens = T <= 16 ? 16 : T <= 32 ? 32 : 64;
  const int64_t tiles = (N + FM - 1) / FM * ((T + f.tokens - 1) / f.tokens), k_blocks = (K + BK - 1) / BK;
  // As many CTAs per cluster as leave one round of two CTAs per SM (one and a half where x is
  // narrow and a CTA little but reads: there more CTAs only add joins), two K blocks each.
  const int64_t most = f.tokens <= 32 ? sms * 3 / 2 : sms * 2;
  f.split = 1;
  for (int sp : {2, 3, 4, 6, 8})
    if (tiles * sp <= most && k_blocks >= 2 * sp) f.split = sp;
  f.one_round = tiles <= 2 * sms;
  // Cycles: the K blocks an SM loads at 64 bytes a cycle, and what a launch costs besides.
  const int64_t per_sm = (tiles * f.split + sms - 1) / sms;
  f.cycles = 9000 + per_sm * ((k_blocks + f.split - 1) / f.split) * (W_BYTES + f.tokens * BK * 2) / 64;
  return f;
}

cudaError_t launch_linear_few(const LinearGemm& g, cudaStream_t s) {
  return g.out_dtype == MOE_F32 ? launch_act<float>(g, s) : launch_act<__nv_bfloat16>(g, s);
}

}  // namespace moe
