// Matrix products of the dense projections on CTA pairs: tcgen05 with cta_group::2, TMA-fed.
//
//   forward  y  = act(x W^T + b) + r   A = x (K-major),       B = W (K-major)
//   dx          = dz W                 A = dz (K-major),      B = W (MN-major)
//   dW          = dz^T x               A = dz (MN-major),     B = x (MN-major)
//
// A cluster of two CTAs computes a 256 x 256 tile: the even CTA issues M = 256, N = 256 MMAs
// whose A rows and B columns are split between the two CTAs' shared memory, so each CTA loads
// 32 KB per 64-wide K block (64 bytes a cycle at the MMA rate, which L2 sustains; a one-SM
// 128 x 128 tile would need twice that).  The ring has three stages of two K blocks: the
// issuer waits once per eight MMAs.  Accumulators are double buffered in TMEM, so the epilogue
// of one tile runs beside the products of the next.  Ragged edges need no masks: TMA fills
// what lies past an operand with zeros, and clips what lies past the output.
//
// Epilogue (four warps per CTA, a lane per row): 128 bytes of each of 32 rows at a time go
// through a swizzled staging block: the residual's block arrives there by TMA while the
// previous one is worked on, is replaced in place by act(z) + r, and leaves by a TMA store.
// An output, residual or pre whose rows do not start on 16-byte boundaries is moved by the
// lanes instead, coalesced along the rows.
//
// Every wait is bounded; a wait that runs out records MOE_ERR_TIMEOUT and the CTA waits for
// what it issued before it frees its TMEM.
#include <algorithm>

#include "activation.cuh"
#include "linear.h"

namespace moe {
namespace {

constexpr int BM = 256, BN = 256;          // pair tile
constexpr int HALF = 128;                  // rows of A, columns of B per CTA
constexpr int BK = 64;
constexpr int STAGES = 3;
constexpr int BLOCK_BYTES = HALF * BK * 2; // one operand, one K block, one CTA
constexpr int STAGE_BYTES = 4 * BLOCK_BYTES;   // two K blocks of A and B
constexpr int STAGING_BYTES = 4096;        // 32 rows of 128 bytes
constexpr int EPI_WARPS = 4;
constexpr int EPI_BYTES = EPI_WARPS * 2 * STAGING_BYTES;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 100000000ull;
constexpr int GROUP_M = 8;                 // row tiles that share the column tiles in flight

struct Args {
  int32_t M, N, K;
  int32_t m_tiles, n_tiles;
  int32_t act;
  const float* bias;
  const void* residual;
  void* pre;
  void* C;
  int64_t ldr, ldc;
  bool tma_r, tma_pre, tma_c;
  int32_t* status;
};

// Tile t: groups of GROUP_M row tiles; within one, the row tiles of a column tile together, so
// the tiles in flight are about as many rows as columns wide and their operands stay in L2.
__device__ __forceinline__ void tile_at(const Args& a, int64_t t, int& m, int& n) {
  const int64_t per = static_cast<int64_t>(GROUP_M) * a.n_tiles;
  const int first = static_cast<int>(t / per) * GROUP_M;
  const int rows = min(GROUP_M, a.m_tiles - first);
  const int in = static_cast<int>(t - (t / per) * per);
  m = first + in % rows;
  n = in / rows;
}

template <typename OUT> struct Piece;      // 16 bytes of an output row
template <> struct Piece<float> {
  static constexpr int N = 4;
  __device__ static void add(float (&y)[4], uint4 r) {
    y[0] += __uint_as_float(r.x);
    y[1] += __uint_as_float(r.y);
    y[2] += __uint_as_float(r.z);
    y[3] += __uint_as_float(r.w);
  }
  __device__ static uint4 pack(const float (&y)[4]) {
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                      __float_as_uint(y[3]));
  }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void add(float (&y)[8], uint4 r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] += __uint_as_float(w[i] << 16);
      y[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
  }
};

// Element e of row r in a swizzled staging block.
template <typename OUT>
__device__ __forceinline__ OUT* staged(uint8_t* blk, int r, int e) {
  constexpr int N = Piece<OUT>::N;
  return reinterpret_cast<OUT*>(blk + r * 128 + (((e / N) ^ (r & 7)) * 16)) + e % N;
}

template <bool A_MN, bool B_MN, typename OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                       const __grid_constant__ CUtensorMap tmP, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* epi = smem + STAGES * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + EPI_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* rbar = tempty + 2;             // [EPI_WARPS][2] residual blocks
  uint64_t* drain = rbar + 2 * EPI_WARPS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* never = const_cast<int*>(abort_flag) + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t smem_base = smem_u32(smem);
  const int64_t pair_id = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int64_t tiles = static_cast<int64_t>(args.m_tiles) * args.n_tiles;
  const int k_blocks = (args.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 2 * EPI_WARPS);
    }
    for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(smem_u32(&rbar[i]), 1);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *never = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), TMEM_COLS);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ---------------------------------------------------------- producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued_parity[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
      bool ok = true;
      for (int64_t t = pair_id; ok && t < tiles; t += n_pairs) {
        int m, n;
        tile_at(args, t, m, n);
        const int m0 = m * BM + static_cast<int>(rank) * HALF;
        const int n0 = n * BN + static_cast<int>(rank) * HALF;
        for (int kb = 0; kb < k_blocks; kb += 2) {
          if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.status,
                                 kWaitLimitNs)) {
            ok = false;
            break;
          }
          const int subs = min(2, k_blocks - kb);
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * subs * 2 * BLOCK_BYTES);
          for (int u = 0; u < subs; ++u) {
            const uint32_t sA = smem_base + stage * STAGE_BYTES + u * 2 * BLOCK_BYTES;
            const uint32_t sB = sA + BLOCK_BYTES;
            const int k0 = (kb + u) * BK;
            if (A_MN) {
              tma_load_2d_pair(sA, &tmA, m0, k0, fb);
              tma_load_2d_pair(sA + kMnLbo, &tmA, m0 + 64, k0, fb);
            } else {
              tma_load_2d_pair(sA, &tmA, k0, m0, fb);
            }
            if (B_MN) {
              tma_load_2d_pair(sB, &tmB, n0, k0, fb);
              tma_load_2d_pair(sB + kMnLbo, &tmB, n0 + 64, k0, fb);
            } else {
              tma_load_2d_pair(sB, &tmB, k0, n0, fb);
            }
          }
          issued_parity[stage] = static_cast<int>(phase);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && leader)
        for (int s = 0; s < STAGES; ++s)
          if (issued_parity[s] >= 0)
            mbar_wait_bounded(smem_u32(&full[s]), static_cast<uint32_t>(issued_parity[s]), never,
                              nullptr, kDrainLimitNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer (even CTA)
    if (leader && lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(BM, BN) | (A_MN ? (1u << 15) : 0u) |
                                 (B_MN ? (1u << 16) : 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int64_t local = 0;
      for (int64_t t = pair_id; ok && t < tiles; t += n_pairs, ++local) {
        const int buf = static_cast<int>(local & 1);
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        if (!mbar_wait_bounded(smem_u32(&tempty[buf]), (use & 1u) ^ 1u, abort_flag, args.status,
                               kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_acc = tmem_base + static_cast<uint32_t>(buf * BN);
        for (int kb = 0; kb < k_blocks; kb += 2) {
          if (!mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, args.status,
                                 kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int subs = min(2, k_blocks - kb);
          for (int u = 0; u < subs; ++u) {
            const uint32_t sA = smem_base + stage * STAGE_BYTES + u * 2 * BLOCK_BYTES;
            const uint32_t sB = sA + BLOCK_BYTES;
#pragma unroll
            for (int j = 0; j < BK / 16; ++j) {
              const uint64_t ad = A_MN ? sw128_mnmajor_desc(sA + j * 2048) : sw128_kmajor_desc(sA) + 2 * j;
              const uint64_t bd = B_MN ? sw128_mnmajor_desc(sB + j * 2048) : sw128_kmajor_desc(sB) + 2 * j;
              tc_mma_bf16_pair(d_acc, ad, bd, idesc, (kb > 0 || u > 0 || j > 0) ? 1u : 0u);
            }
          }
          tc_commit_pair(smem_u32(&empty[stage]), 0x3);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(smem_u32(&tfull[buf]), 0x3);
      }
      if (!ok) {
        tc_commit_pair(smem_u32(drain), 0x1);
        mbar_wait_bounded(smem_u32(drain), 0, never, nullptr, kDrainLimitNs);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue (both CTAs)
    constexpr int CW = 128 / static_cast<int>(sizeof(OUT));   // columns of a staging block
    constexpr int CHUNKS = BN / CW;
    constexpr int PN = Piece<OUT>::N;
    const int q = warp & 3;                  // TMEM lanes of this warp
    uint8_t* blk0 = epi + (warp - 2) * 2 * STAGING_BYTES;
    uint64_t* bars = rbar + 2 * (warp - 2);
    const bool res = args.residual != nullptr, pre = args.pre != nullptr;
    uint32_t rphase = 0, inflight = 0;      // a bit per staging block; residual blocks on their way
    int64_t local = 0;
    bool ok = true;
    for (int64_t t = pair_id; ok && t < tiles; t += n_pairs, ++local) {
      int m, n;
      tile_at(args, t, m, n);
      const int buf = static_cast<int>(local & 1);
      const uint32_t use = static_cast<uint32_t>(local >> 1);
      const int64_t row0 = static_cast<int64_t>(m) * BM + rank * HALF + q * 32;
      const int rows = static_cast<int>(min(static_cast<int64_t>(32), args.M - row0));   // <= 0: none
      // Residual block of chunk c into staging block b, once the stores from it have been read.
      auto load_residual = [&](int c, int b) {
        inflight |= 1u << b;
        if (lane == 0) {
          bulk_wait_read<0>();
          mbar_arrive_expect_tx(smem_u32(&bars[b]), STAGING_BYTES);
          tma_load_2d(smem_u32(blk0 + b * STAGING_BYTES), &tmR, n * BN + c * CW,
                      static_cast<int32_t>(row0), smem_u32(&bars[b]));
        }
      };
      const bool tma_res = res && args.tma_r && rows > 0;
      if (tma_res) load_residual(0, 0);
      bool ready = true;
      if (lane == 0)
        ready = mbar_wait_bounded(smem_u32(&tfull[buf]), use & 1u, abort_flag, args.status, kWaitLimitNs);
      ok = __shfl_sync(0xffffffffu, ready ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(buf * BN);
      if (rows > 0) {
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
          const int col = n * BN + c * CW;
          if (col >= args.N) break;
          const int cols = min(CW, args.N - col);
          // y uses the two blocks in turn, or block 0 beside a pre in block 1
          const int yb = pre ? 0 : c & 1;
          uint8_t* yblk = blk0 + yb * STAGING_BYTES;
          uint8_t* pblk = blk0 + STAGING_BYTES;
          uint32_t va[32], vb[32];
          if (CW == 64)
            tmem_ld32x2(taddr + c * CW, taddr + c * CW + 32, va, vb);
          else
            tmem_ld32(taddr + c * CW, va);
          if (tma_res) {
            if (pre) {
              if (c > 0) load_residual(c, 0);
            } else if (c + 1 < CHUNKS && col + CW < args.N) {
              load_residual(c + 1, (c + 1) & 1);
            }
            const bool here =
                mbar_wait_bounded(smem_u32(&bars[yb]), (rphase >> yb) & 1u, abort_flag, args.status, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, here);
            if (!ok) break;
            rphase ^= 1u << yb;
            inflight &= ~(1u << yb);
          } else {
            // the stores that left from the blocks about to be written have been read
            if (lane == 0) {
              if (pre) bulk_wait_read<0>(); else bulk_wait_read<1>();
            }
            __syncwarp();
            if (res) {
              const OUT* r = static_cast<const OUT*>(args.residual) + row0 * args.ldr + col;
              for (int i = lane; i < rows * CW; i += 32) {
                const int rr = i / CW, e = i % CW;
                if (e < cols) *staged<OUT>(yblk, rr, e) = r[rr * args.ldr + e];
              }
              __syncwarp();
            }
          }
#pragma unroll
          for (int j = 0; j < CW / PN; ++j) {
            float z[PN];
#pragma unroll
            for (int e = 0; e < PN; ++e) {
              const int i = j * PN + e;
              z[e] = __uint_as_float(i < 32 ? va[i & 31] : vb[i & 31]);
              if (args.bias != nullptr && i < cols) z[e] += __ldg(args.bias + col + i);
            }
            const int off = lane * 128 + ((j ^ (lane & 7)) * 16);
            if (pre) *reinterpret_cast<uint4*>(pblk + off) = Piece<OUT>::pack(z);
            if (args.act != MOE_ACT_NONE) {
#pragma unroll
              for (int e = 0; e < PN; ++e) z[e] = act_value(z[e], args.act);
            }
            if (res) Piece<OUT>::add(z, *reinterpret_cast<const uint4*>(yblk + off));
            *reinterpret_cast<uint4*>(yblk + off) = Piece<OUT>::pack(z);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && (args.tma_c || (pre && args.tma_pre))) {
            if (args.tma_c) tma_store_2d(&tmC, col, static_cast<int32_t>(row0), smem_u32(yblk));
            if (pre && args.tma_pre) tma_store_2d(&tmP, col, static_cast<int32_t>(row0), smem_u32(pblk));
            bulk_commit();
          }
          if (!args.tma_c) {
            OUT* y = static_cast<OUT*>(args.C) + row0 * args.ldc + col;
            for (int i = lane; i < rows * CW; i += 32) {
              const int rr = i / CW, e = i % CW;
              if (e < cols) y[rr * args.ldc + e] = *staged<OUT>(yblk, rr, e);
            }
          }
          if (pre && !args.tma_pre) {
            OUT* p = static_cast<OUT*>(args.pre) + row0 * args.N + col;
            for (int i = lane; i < rows * CW; i += 32) {
              const int rr = i / CW, e = i % CW;
              if (e < cols) p[rr * static_cast<int64_t>(args.N) + e] = *staged<OUT>(pblk, rr, e);
            }
          }
          __syncwarp();   // the staging blocks have been read
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
    }
    if (lane == 0) {
      for (int b = 0; b < 2; ++b)
        if ((inflight >> b) & 1u)   // only after a wait ran out
          mbar_wait_bounded(smem_u32(&bars[b]), (rphase >> b) & 1u, never, nullptr, kDrainLimitNs);
      bulk_wait_all();   // the output blocks are written
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // no CTA leaves while its partner may still use its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 8 * (2 * STAGES + 4 + 2 * EPI_WARPS + 1) + 32;

bool rows16(const void* p, int64_t ld, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % (dtype == MOE_F32 ? 4 : 8) == 0;
}

template <bool A_MN, bool B_MN, typename OUT>
cudaError_t launch_typed(const LinearGemm& g, cudaStream_t s) {
  constexpr int32_t dt = sizeof(OUT) == 4 ? MOE_F32 : MOE_BF16;
  constexpr uint32_t cw = 128 / sizeof(OUT);
  Args a{};
  a.M = static_cast<int32_t>(g.M);
  a.N = g.N;
  a.K = g.K;
  a.m_tiles = static_cast<int32_t>((g.M + BM - 1) / BM);
  a.n_tiles = (g.N + BN - 1) / BN;
  a.act = g.act;
  a.bias = g.bias;
  a.residual = g.residual;
  a.pre = g.pre;
  a.C = g.C;
  a.ldr = g.ldr;
  a.ldc = g.ldc;
  a.status = g.status;
  a.tma_c = rows16(g.C, g.ldc, dt);
  a.tma_r = g.residual && rows16(g.residual, g.ldr, dt);
  a.tma_pre = g.pre && rows16(g.pre, g.N, dt);
  CUtensorMap mA, mB, mC, mR, mP;
  const uint64_t M = static_cast<uint64_t>(g.M), N = g.N, K = g.K;
  if (!(A_MN ? make_strided_map(&mA, MOE_BF16, g.A, M, K, g.lda, 64, BK)
             : make_strided_map(&mA, MOE_BF16, g.A, K, M, g.lda, BK, HALF)) ||
      !(B_MN ? make_strided_map(&mB, MOE_BF16, g.B, N, K, g.ldb, 64, BK)
             : make_strided_map(&mB, MOE_BF16, g.B, K, N, g.ldb, BK, HALF)))
    return cudaErrorInvalidValue;
  mC = mR = mP = mA;
  if ((a.tma_c && !make_strided_map(&mC, dt, g.C, N, M, g.ldc, cw, 32)) ||
      (a.tma_r && !make_strided_map(&mR, dt, g.residual, N, M, g.ldr, cw, 32)) ||
      (a.tma_pre && !make_strided_map(&mP, dt, g.pre, N, M, N, cw, 32)))
    return cudaErrorInvalidValue;
  auto kern = linear_pair_kernel<A_MN, B_MN, OUT>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
  const int64_t pairs = std::min<int64_t>(tiles, std::max(1, device_sm_count() / 2));
  kern<<<static_cast<unsigned>(2 * pairs), THREADS, kSmemBytes, s>>>(mA, mB, mC, mR, mP, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_pair(const LinearGemm& g, cudaStream_t s) {
  const bool f32 = g.out_dtype == MOE_F32;
  if (g.a_mn)
    return f32 ? launch_typed<true, true, float>(g, s) : launch_typed<true, true, __nv_bfloat16>(g, s);
  if (g.b_mn)
    return f32 ? launch_typed<false, true, float>(g, s) : launch_typed<false, true, __nv_bfloat16>(g, s);
  return f32 ? launch_typed<false, false, float>(g, s) : launch_typed<false, false, __nv_bfloat16>(g, s);
}

}  // namespace moe
