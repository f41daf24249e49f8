// Matrix products of the dense projections on CTA pairs: tcgen05 with cta_group::2, TMA-fed.
//
//   forward  y  = act(x W^T + b) + r   A = x (K-major),       B = W (K-major)
//   dx          = dz W                 A = dz (K-major),      B = W (MN-major)
//   dW          = dz^T x               A = dz (MN-major),     B = x (MN-major)
//
// A cluster of two CTAs computes a 256 x 256 tile: the even CTA issues M = 256, N = 256 MMAs
// whose A rows and B columns are split between the two CTAs' shared memory, so each CTA loads
// 32 KB per 64-wide K block (64 bytes a cycle at the MMA rate, which is what L2 sustains; 128
// columns need 96 and run at two thirds of the rate).  Accumulators are double buffered in TMEM, so the epilogue
// of one tile runs beside the products of the next.  Ragged edges need no masks: TMA fills
// what lies past an operand with zeros, and clips what lies past the output.
//
// Tiles rarely fill whole rounds of 76 pairs.  Where the last, partial round would leave enough
// of them idle, its tiles are cut along the depth into equal parts for as many pairs: each leaves
// its partial sums (fp32) in scratch memory, and the CTA that finds itself the last of a tile
// adds the parts in their order along K, whoever came last, so the result does not depend on
// it.  The cut tiles come first: the joining runs beside the products of the whole tiles.
// Otherwise, where the partial round of a bf16 output has at most half as many tiles as there are
// pairs, each is shared by two pairs as tiles of 128 columns: half the epilogue, and the products
// in about three quarters of the time (a narrow tile needs 96 bytes a cycle, more than an SM
// gets).  1237 x 2048 x 5632: 26.4 -> 24.7 us, with GELU 29.8 -> 27.7 us; 8192 x 2560 x 2560:
// 67.4 -> 65.8 us.  Kernels without narrow tiles are built apart: the width is a constant there
// (1 to 2 % of 16384 x 2048 x 5632).
//
// Epilogue: eight warps per CTA (two per TMEM lane quarter, half of the columns each), a lane per
// row.  The residual's blocks of 32 rows come by TMA into swizzled shared memory, two per warp,
// the first while the tile's products still run.
//   fp32 outputs: blocks of 128-byte rows, replaced in place by act(z) + r, leave by 32-byte
//     stores that each cover 128 neighbouring bytes of eight rows (an 84 MB output written by a lane
//     per row takes 25 us, so 16.5 us, in whole 512-byte rows 14.6 us); 8192 x 2560 x 2560 with
//     residual 112 us against 135 with a lane per row.  The blocks leave room for a ring of five K
//     blocks.
//   bf16 outputs: half the bytes.  64-byte rows, stored by a lane per row in 32-byte sectors, leave
//     room for three ring stages of two K blocks, so that the issuer waits once per eight MMAs
//     (8192 x 2560 x 2560 in 69.5 us; with five or six stages of one 72 to 75 us).
// A matrix whose rows are not aligned to 16 bytes is moved element by element along the rows, in
// kernels of their own: the epilogue runs once per tile and is bound by fetching its code, so
// it holds no path that a launch does not take (5 % of 8192 x 2560 x 2560) and loops rather than
// unrolls.
//
// The tensor core drops the bits of an addition that do not fit fp32 instead of rounding, an
// error that grows with the length of the sum and has one sign (measured 2.7e-6 of the result
// at a depth of 2560).  bf16 outputs do not see it.  For fp32 outputs a sum is taken in segments
// of at most 896: each ends in its own TMEM buffer and the epilogue adds them in registers, rounded.
//
// Every wait is bounded; a wait that runs out records MOE_ERR_TIMEOUT and the CTA waits for
// what it issued before it frees its TMEM.
#include <algorithm>

#include "activation.cuh"
#include "linear.h"

namespace moe {
namespace {

constexpr int BM = 256;                    // rows of a pair tile
constexpr int HALF = 128;                  // rows of A per CTA
constexpr int BK = 64;
constexpr int A_BYTES = HALF * BK * 2;     // one K block, one CTA
constexpr int EPI_WARPS = 8;
constexpr int F32_SEGMENT = 14;            // most K blocks of one fp32 partial sum
constexpr int EPI_WARP0 = 4;               // warps 0, 1: producer, issuer; a warpgroup of their own
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// What depends on the tile's width and the output type.
template <int BN, bool F32> struct Tile {
  static constexpr int COLS = BN / 2;                      // columns of B per CTA, and of an epilogue warp
  static constexpr int B_BYTES = COLS * BK * 2;
  static constexpr int SUB_BYTES = A_BYTES + B_BYTES;      // one K block of A and B
  static constexpr int SUBS = F32 ? 1 : 2;                 // K blocks of a ring stage
  static constexpr int STAGE_BYTES = SUBS * SUB_BYTES;
  static constexpr int STAGES = F32 ? (BN == 256 ? 5 : 6) : (BN == 256 ? 3 : 4);
  static constexpr int ROW_BYTES = F32 ? 128 : 64;         // of an output block
  static constexpr int BLOCK_BYTES = 32 * ROW_BYTES;
  static constexpr int EPI_BYTES = EPI_WARPS * 2 * BLOCK_BYTES;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 8 * (2 * STAGES + 4 + 2 * EPI_WARPS + 1) + 32;
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};
// Registers of the epilogue's threads and of the others, within the 384 x 168 of the launch; the
// epilogue of fp32 outputs holds 128 sums.
template <bool F32> struct Regs {
  static constexpr int EPI = F32 ? 224 : 208, OTHER = F32 ? 56 : 80;
  static_assert(32 * (EPI_WARPS * EPI + EPI_WARP0 * OTHER) <= THREADS * 168, "register split");
};
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 100000000ull;
constexpr int GROUP_M = 8;                 // row tiles that share the column tiles in flight

struct Args {
  int32_t M, N, K;
  int32_t m_tiles, n_tiles;
  int32_t cut_tiles;        // tiles 0 .. cut_tiles - 1 are cut along K
  int32_t parts;            // into this many parts; pair r parts + k holds part k of tile r
  int64_t whole;            // NARROW: tiles past this one are two narrow ones each
  const float* part;        // partial sums of db
  float* db;
  int64_t db_parts;
  int32_t db_cols;
  const float* bias;
  const void* residual;
  void* pre;
  void* C;
  int64_t ldr, ldc;
  int32_t act;              // of kActAny
  int32_t al_pre, al_c;     // bytes the rows are aligned to: 32, 16, or 0 (less)
  int32_t* status;
  float* scratch;
  unsigned* tickets;
};

// One piece of a pair's work: K blocks [kb0, kb1) of tile (m, n).
struct Item {
  int m, n, kb0, kb1;
  int first, cols;          // NARROW: of the tile's columns: 0, 256, or one half of them
  int parts;                // parts of this tile; 1: the whole tile
  int cut;                  // index of the cut tile
};

// Item i of a pair; false past the last.  A pair's part of a cut tile comes first, a narrow tile
// last.
// Tiles are numbered in groups of GROUP_M row tiles, within one the row tiles of a column tile
// together, so that the tiles in flight are about as many rows as columns wide and their
// operands stay in L2.
template <bool NARROW>
__device__ __forceinline__ bool item_at(const Args& a, int pair, int n_pairs, int i, Item& o) {
  const int k_blocks = (a.K + BK - 1) / BK;
  int64_t t;
  if (pair < a.cut_tiles * a.parts && i == 0) {
    // parts of whole ring stages (two K blocks)
    const int stages = (k_blocks + 1) / 2, k = pair % a.parts;
    o.parts = a.parts;
    o.cut = pair / a.parts;
    o.kb0 = static_cast<int>(static_cast<int64_t>(stages) * k / a.parts) * 2;
    o.kb1 = min(static_cast<int>(static_cast<int64_t>(stages) * (k + 1) / a.parts) * 2, k_blocks);
    t = o.cut;
  } else {
    o.parts = 1;
    o.kb0 = 0;
    o.kb1 = k_blocks;
    t = a.cut_tiles + pair + static_cast<int64_t>(pair < a.cut_tiles * a.parts ? i - 1 : i) * n_pairs;
  }
  o.first = 0;
  o.cols = 256;
  if (NARROW && t >= a.whole) {   // narrow tiles t - whole: the halves of whole, whole + 1, ...
    const int64_t h = t - a.whole;
    t = a.whole + h / 2;
    o.first = static_cast<int>(h % 2) * 128;
    o.cols = 128;
  }
  if (t >= static_cast<int64_t>(a.m_tiles) * a.n_tiles) return false;
  const int64_t per = static_cast<int64_t>(GROUP_M) * a.n_tiles;
  const int first = static_cast<int>(t / per) * GROUP_M;
  const int rows = min(GROUP_M, a.m_tiles - first);
  const int in = static_cast<int>(t - (t / per) * per);
  o.m = first + in % rows;
  o.n = in / rows;
  return true;
}

// K blocks of one accumulation: all, or for fp32 outputs equal segments of at most F32_SEGMENT.
template <bool SEGMENTED>
__device__ __forceinline__ int segment_blocks(const Item& it) {
  const int blocks = it.kb1 - it.kb0;
  if (!SEGMENTED) return blocks;
  const int n = (blocks + F32_SEGMENT - 1) / F32_SEGMENT;
  return (blocks + n - 1) / n;
}

// Barrier of the epilogue warps that tells whether `ok` holds in all of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "n"(32 * EPI_WARPS)
      : "memory");
  return all != 0;
}

template <typename OUT> struct Row64;      // CW values as 16 words
template <> struct Row64<float> {
  static constexpr int CW = 16;
  __device__ __forceinline__ static void add(float (&z)[16], const uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] += __uint_as_float(w[i]);
  }
  __device__ __forceinline__ static void pack(const float (&z)[16], uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(z[i]);
  }
};
template <> struct Row64<__nv_bfloat16> {
  static constexpr int CW = 32;
  __device__ __forceinline__ static void add(float (&z)[32], const uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      z[2 * i] += __uint_as_float(w[i] << 16);
      z[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static void pack(const float (&z)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(z[2 * i], z[2 * i + 1]);
  }
};

// 64 bytes of a row, 16 words, to global memory; of a ragged last step the `pieces` (of four) that
// exist.
__device__ __forceinline__ void store64(void* p, int align, int pieces, const uint32_t (&w)[16]) {
  if (align == 32 && pieces == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<char*>(p) + 32 * h),
                   "r"(w[8 * h]), "r"(w[8 * h + 1]), "r"(w[8 * h + 2]), "r"(w[8 * h + 3]), "r"(w[8 * h + 4]),
                   "r"(w[8 * h + 5]), "r"(w[8 * h + 6]), "r"(w[8 * h + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (h < pieces)
        static_cast<uint4*>(p)[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
  }
}

// The 16-byte piece j of row r of a block, in the swizzle of its row width (so that neither a lane
// per row nor four lanes per row collide).
template <typename OUT>
__device__ __forceinline__ uint4* block_piece(uint8_t* blk, int r, int j) {
  return sizeof(OUT) == 4 ? reinterpret_cast<uint4*>(blk + r * 128 + ((j ^ (r & 7)) * 16))
                          : reinterpret_cast<uint4*>(blk + r * 64 + ((j ^ ((r >> 1) & 3)) * 16));
}
template <typename OUT>
__device__ __forceinline__ OUT* block_element(uint8_t* blk, int r, int e) {
  constexpr int N = 16 / static_cast<int>(sizeof(OUT));
  return reinterpret_cast<OUT*>(block_piece<OUT>(blk, r, e / N)) + e % N;
}

// The rows x cols (of 32: 128 bytes of fp32, 64 of bf16) of a block that exist, ld elements apart
// from p on, to memory.  Called by the whole warp after a __syncwarp.  ALIGNED: fp32 only.
template <typename OUT, bool ALIGNED>
__device__ __forceinline__ void store_block(OUT* p, int64_t ld, int align, int rows, int cols, int lane, uint8_t* blk) {
  if constexpr (ALIGNED) {
    const int q = lane % 4;                       // 32 bytes of the row
    const int pieces = cols / 4 - 2 * q;          // that exist, from q on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + lane / 4;
      const uint4 u = *block_piece<OUT>(blk, r, 2 * q), v = *block_piece<OUT>(blk, r, 2 * q + 1);
      OUT* at = p + r * ld + 8 * q;
      if (r < rows && pieces >= 2 && align == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(u.x), "r"(u.y),
                     "r"(u.z), "r"(u.w), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
      } else if (r < rows && pieces > 0) {
        reinterpret_cast<uint4*>(at)[0] = u;
        if (pieces >= 2) reinterpret_cast<uint4*>(at)[1] = v;
      }
    }
  } else if (lane < cols) {
#pragma unroll 8
    for (int r = 0; r < rows; ++r) p[r * ld + lane] = *block_element<OUT>(blk, r, lane);
  }
}
// The same from memory, a column per lane, every row on its way at once: fp32 by asynchronous
// copies (through registers the epilogue's sums leave too few), bf16 through registers.
template <typename OUT>
__device__ __forceinline__ void load_block(const OUT* p, int64_t ld, int rows, int cols, int lane, uint8_t* blk) {
  if constexpr (sizeof(OUT) == 4) {
    if (lane < cols) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(block_element<OUT>(blk, r, lane))),
                     "l"(p + r * ld + lane)
                     : "memory");
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else {
    OUT v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r)
      if (r < rows && lane < cols) v[r] = p[r * ld + lane];
#pragma unroll
    for (int r = 0; r < 32; ++r)
      if (r < rows && lane < cols) *block_element<OUT>(blk, r, lane) = v[r];
  }
}

constexpr int kActAny = -1;
template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
#define MOE_CALL(ACT) [&]() { _Pragma("unroll") for (int e = 0; e < N; ++e) z[e] = act_value<ACT>(z[e]); }()
  MOE_DISPATCH_ACT(act, MOE_CALL)
#undef MOE_CALL
}

// Columns of db by the warps that neither load nor multiply: eight columns of a warp at a time, four
// lanes to a column, each lane four running sums (adds of fixed order).  It saves a launch before
// the products: gradients of 999 x 2048 to 1407 30.8 -> 29.5 us, of 500 x 700 to 999 in fp32 33.1 ->
// 30.0, of 8192 x 2560 x 2560 155.4 -> 153.3.
__device__ __forceinline__ void sum_parts(const Args& a, int warp, int warps, int lane) {
  const int parts = static_cast<int>(a.db_parts);
  const int64_t step = static_cast<int64_t>(a.db_cols) * 4;
#pragma unroll 1
  for (int c0 = warp * 8; c0 < a.db_cols; c0 += warps * 8) {
    const int c = min(c0 + lane % 8, a.db_cols - 1);   // past the end: the last column once more
    float v[4] = {};
    const float* p = a.part + static_cast<int64_t>(lane / 8) * a.db_cols + c;
#pragma unroll 1
    for (int b = lane / 8; b < parts; b += 16) {
#pragma unroll
      for (int u = 0; u < 4; ++u, p += step)
        if (b + 4 * u < parts) v[u] += *p;
    }
    float sum = (v[0] + v[1]) + (v[2] + v[3]);
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < 8 && c0 + lane < a.db_cols) a.db[c] = sum;
  }
}

// ALIGNED: every row that the epilogue touches starts on a 16-byte boundary and N ends on one; else
// ACT is kActAny, the run-time activation.
template <int BN, bool A_MN, bool B_MN, typename OUT, int ACT, bool ALIGNED, bool NARROW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmBn, const __grid_constant__ CUtensorMap tmR,
                       const Args args) {
  static_assert(!NARROW || (BN == 256 && !A_MN && !B_MN && sizeof(OUT) == 2), "narrow tiles");
  using TL = Tile<BN, sizeof(OUT) == 4>;
  constexpr int STAGES = TL::STAGES, WARP_COLS = TL::COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* epi = smem + STAGES * TL::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + TL::EPI_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* rbar = tempty + 2;             // [EPI_WARPS][2] residual blocks
  uint64_t* drain = rbar + 2 * EPI_WARPS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* never = const_cast<int*>(abort_flag) + 1;
  int* last_part = never + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t smem_base = smem_u32(smem);
  const int pair_id = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);
  constexpr bool SEGMENTED = sizeof(OUT) == 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 2 * EPI_WARPS);   // of both CTAs
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
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), TL::TMEM_COLS);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  launch_dependents();
  wait_for_previous();

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<SEGMENTED>::OTHER));
    if (warp == 0) {
      // ---------------------------------------------------------- producer (both CTAs)
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        int issued_parity[STAGES];
#pragma unroll
        for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
        bool ok = true;
        Item it;
        for (int i = 0; ok && item_at<NARROW>(args, pair_id, n_pairs, i, it); ++i) {
          const int m0 = it.m * BM + static_cast<int>(rank) * HALF;
          const int cols = NARROW ? it.cols / 2 : TL::COLS;   // of this CTA
          const int n0 = it.n * BN + it.first + static_cast<int>(rank) * cols;
          const uint32_t sub_bytes = A_BYTES + cols * BK * 2;
          for (int kb = it.kb0; kb < it.kb1; kb += TL::SUBS) {
            if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, args.status,
                                   kWaitLimitNs)) {
              ok = false;
              break;
            }
            const int subs = min(TL::SUBS, it.kb1 - kb);
            const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
            if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * subs * sub_bytes);
            for (int u = 0; u < subs; ++u) {
              const uint32_t sA = smem_base + stage * TL::STAGE_BYTES + u * TL::SUB_BYTES;
              const uint32_t sB = sA + A_BYTES;
              const int k0 = (kb + u) * BK;
              if (A_MN) {
                tma_load_2d_pair(sA, &tmA, m0, k0, fb);
                tma_load_2d_pair(sA + kMnLbo, &tmA, m0 + 64, k0, fb);
              } else {
                tma_load_2d_pair(sA, &tmA, k0, m0, fb);
              }
              if (B_MN) {
                tma_load_2d_pair(sB, &tmB, n0, k0, fb);
                if (TL::COLS > 64) tma_load_2d_pair(sB + kMnLbo, &tmB, n0 + 64, k0, fb);
              } else {
                tma_load_2d_pair(sB, NARROW && it.cols != BN ? &tmBn : &tmB, k0, n0, fb);
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
        constexpr uint32_t major = (A_MN ? (1u << 15) : 0u) | (B_MN ? (1u << 16) : 0u);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t fill = 0;                     // TMEM buffers filled
        Item it;
        for (int i = 0; ok && item_at<NARROW>(args, pair_id, n_pairs, i, it); ++i) {
          const int seg = segment_blocks<SEGMENTED>(it);
          const uint32_t idesc = (NARROW && it.cols != BN ? idesc_bf16_f32(BM, BN / 2) : idesc_bf16_f32(BM, BN)) | major;
          for (int s0 = it.kb0; ok && s0 < it.kb1; s0 += seg, ++fill) {
            const int s1 = min(s0 + seg, it.kb1);
            const uint32_t d_acc = tmem_base + (fill & 1) * BN;
            ok = mbar_wait_bounded(smem_u32(&tempty[fill & 1]), ((fill >> 1) & 1u) ^ 1u, abort_flag, args.status,
                                   kWaitLimitNs);
            tc_fence_after();
            for (int kb = s0; ok && kb < s1; kb += TL::SUBS) {
              ok = mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, args.status, kWaitLimitNs);
              if (!ok) break;
              tc_fence_after();
              const int subs = min(TL::SUBS, it.kb1 - kb);
              for (int u = 0; u < subs; ++u) {
                const uint32_t sA = smem_base + stage * TL::STAGE_BYTES + u * TL::SUB_BYTES;
                const uint32_t sB = sA + A_BYTES;
#pragma unroll
                for (int j = 0; j < BK / 16; ++j) {
                  const uint64_t ad = A_MN ? sw128_mnmajor_desc(sA + j * 2048) : sw128_kmajor_desc(sA) + 2 * j;
                  const uint64_t bd = B_MN ? sw128_mnmajor_desc(sB + j * 2048) : sw128_kmajor_desc(sB) + 2 * j;
                  tc_mma_bf16_pair(d_acc, ad, bd, idesc, (kb > s0 || u > 0 || j > 0) ? 1u : 0u);
                }
              }
              tc_commit_pair(smem_u32(&empty[stage]), 0x3);
              if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (ok) tc_commit_pair(smem_u32(&tfull[fill & 1]), 0x3);
          }
        }
        if (!ok) {
          tc_commit_pair(smem_u32(drain), 0x1);
          mbar_wait_bounded(smem_u32(drain), 0, never, nullptr, kDrainLimitNs);
        }
      }
    } else if (B_MN && args.db != nullptr) {
      // -------------------------------------------------------- sums of db (warps 2 and 3 of both CTAs)
      sum_parts(args, blockIdx.x * 2 + warp - 2, gridDim.x * 2, lane);
    }
  } else {
    // ---------------------------------------------------------- epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<SEGMENTED>::EPI));
    constexpr int CW = Row64<OUT>::CW;       // columns of 64 bytes
    constexpr int PER = TL::ROW_BYTES / 64;  // of which a block has 2 (fp32) or 1
    constexpr int BCOLS = PER * CW;
    // results go through a block (and pre through the second), or from the registers
    constexpr bool STAGED = SEGMENTED || !ALIGNED;
    const int q = warp & 3;                  // TMEM lanes of this warp
    const int half = (warp - EPI_WARP0) >> 2;   // its columns
    uint8_t* blk = epi + (warp - EPI_WARP0) * 2 * TL::BLOCK_BYTES;
    uint64_t* bars = rbar + 2 * (warp - EPI_WARP0);
    const int bufs = STAGED && args.pre != nullptr ? 1 : 2;   // that y and the residual take in turn
    uint32_t loads = 0, reads = 0;           // residual blocks asked for and read, over all tiles
    const bool res = args.residual != nullptr;
    uint32_t fill = 0;
    bool ok = true;
    Item it;
    // a part of a cut tile is taken up even after a failure: the epilogue warps agree there
    for (int i = 0; item_at<NARROW>(args, pair_id, n_pairs, i, it) && (ok || it.parts > 1); ++i) {
      const int64_t row0 = static_cast<int64_t>(it.m) * BM + rank * HALF + q * 32;
      const int warp_cols = NARROW ? it.cols / 2 : WARP_COLS;   // of this warp
      const int col0 = it.n * BN + it.first + half * warp_cols;
      // rows and columns of this warp's block; none where it lies past the output
      const int rows = col0 < args.N ? static_cast<int>(min(static_cast<int64_t>(32), args.M - row0)) : 0;
      const OUT* rrow = static_cast<const OUT*>(args.residual) + row0 * args.ldr + col0;
      const int blocks = rows > 0 ? min(warp_cols / BCOLS, (args.N - col0 + BCOLS - 1) / BCOLS) : 0;
      const bool tma_res = ALIGNED && res;
      // the residual of block c into the buffer of its turn
      auto load_residual = [&](int c) {
        if (c >= blocks) return;
        const uint32_t b = bufs == 1 ? 0 : loads & 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_u32(&bars[b]), TL::BLOCK_BYTES);
          tma_load_2d(smem_u32(blk + b * TL::BLOCK_BYTES), &tmR, col0 + c * BCOLS, static_cast<int32_t>(row0),
                      smem_u32(&bars[b]));
        }
        ++loads;
      };
      if (tma_res && it.parts == 1)
        for (int c = 0; c < bufs; ++c) load_residual(c);
      // The bias, a column per lane (loaded by every lane for each of its columns it costs more than
      // the rest of an epilogue: 8192 x 512 x 2560 fp32 in 57 us against 40 without it).
      float bias[WARP_COLS / 32];
#pragma unroll
      for (int k = 0; k < WARP_COLS / 32; ++k) {
        const int col = col0 + k * 32 + lane;
        bias[k] = args.bias != nullptr && k * 32 < warp_cols && col < args.N ? args.bias[col] : 0.f;
      }
      // Waits for the next TMEM buffer; its columns of this warp start at taddr.
      uint32_t taddr = 0;
      auto wait_fill = [&]() {
        bool ready = true;
        if (lane == 0)
          ready = mbar_wait_bounded(smem_u32(&tfull[fill & 1]), (fill >> 1) & 1u, abort_flag, args.status,
                                    kWaitLimitNs);
        ready = __shfl_sync(0xffffffffu, ready ? 1 : 0, 0) != 0;
        tc_fence_after();
        taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                static_cast<uint32_t>((fill & 1) * BN + half * warp_cols);
        return ready;
      };
      auto release_fill = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[fill & 1]), 0));
        ++fill;
      };
      // where this warp's lane of a pair's partial sums starts (32 groups of four columns)
      auto slot = [&](int pair) {
        return reinterpret_cast<float4*>(args.scratch) + static_cast<size_t>(pair) * (BM * 256 / 4) +
               (static_cast<size_t>(rank) * EPI_WARPS + (warp - EPI_WARP0)) * (WARP_COLS / 4) * 32 + lane;
      };
      float acc[SEGMENTED ? WARP_COLS : 1];
      // Leaves this part of a cut tile in scratch memory, four columns of a row per access; the
      // last CTA to come puts the parts' sum in this part's place in TMEM.
      enum { kFailed, kNotLast, kJoined };
      auto join = [&]() -> int {
        float4* mine = slot(pair_id);
        if (ok) {
          if (SEGMENTED) {
#pragma unroll
            for (int e = 0; e < WARP_COLS; e += 4) {
              float f[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) f[k] = acc[(e + k) % (SEGMENTED ? WARP_COLS : 1)];
              __stcg(mine + e / 4 * 32, make_float4(f[0], f[1], f[2], f[3]));
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < WARP_COLS; c += 32) {
              uint32_t v[32];
              tmem_ld32(taddr + c, v);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                __stcg(mine + (c + e) / 4 * 32, make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                                            __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])));
            }
          }
        }
        __threadfence();
        if (!epilogue_all(ok)) return kFailed;
        if (warp == EPI_WARP0 && lane == 0) {
          // byte 2 cut + rank of the counts: parts that have arrived
          const int b = 2 * it.cut + static_cast<int>(rank);
          const unsigned before = (atomicAdd(args.tickets + b / 4, 1u << (8 * (b % 4))) >> (8 * (b % 4))) & 0xffu;
          const bool last = static_cast<int>(before) == it.parts - 1;
          if (last) atomicSub(args.tickets + b / 4, static_cast<unsigned>(it.parts) << (8 * (b % 4)));
          *last_part = last ? 1 : 0;
          __threadfence();
        }
        epilogue_all(true);
        const bool last = *reinterpret_cast<volatile int*>(last_part) != 0;
        epilogue_all(true);   // read by all before the next part writes it
        if (!last) return kNotLast;
        __threadfence();
#pragma unroll 1
        for (int c = 0; c < WARP_COLS; c += 32) {
          float sum[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[e] = 0.f;
#pragma unroll 4
          for (int k = 0; k < it.parts; ++k) {
            const float4* p = slot(it.cut * it.parts + k) + c / 4 * 32;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 w = __ldcg(p + e * 32);
              sum[4 * e] += w.x;
              sum[4 * e + 1] += w.y;
              sum[4 * e + 2] += w.z;
              sum[4 * e + 3] += w.w;
            }
          }
          uint32_t v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(sum[e]);
          tmem_st32(taddr + c, v);
        }
        return kJoined;
      };
      if (SEGMENTED) {
        // All segments but the last into registers, each buffer free again at once; the last one's
        // buffer takes the sum, so that what follows can loop over it (unrolled over registers it
        // is bound by fetching its own code: 8192 x 2560 x 2560 with GELU 223 us).
        const int seg = segment_blocks<SEGMENTED>(it);
        for (int s0 = it.kb0; ok && s0 < it.kb1; s0 += seg) {
          ok = wait_fill();
          if (!ok) break;
          const bool first = s0 == it.kb0, last = s0 + seg >= it.kb1;
          if (first && last && it.parts == 1) break;   // one segment: its buffer holds the sum
#pragma unroll
          for (int k = 0; k < WARP_COLS; k += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + k, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float& sum = acc[(k + e) % (SEGMENTED ? WARP_COLS : 1)];
              sum = (first ? 0.f : sum) + __uint_as_float(v[e]);
              v[e] = __float_as_uint(sum);
            }
            if (last && it.parts == 1) tmem_st32(taddr + k, v);
          }
          if (!last) release_fill();
        }
      } else if (ok) {
        ok = wait_fill();
      }
      int joined = kJoined;
      if (it.parts > 1) {
        joined = join();
        ok = joined != kFailed;
        if (joined == kNotLast) release_fill();
      }
      if (!ok) break;
      if (joined == kNotLast) continue;
      if (tma_res && it.parts > 1)
        for (int c = 0; c < bufs; ++c) load_residual(c);
#pragma unroll 1
      for (int c = 0; c < warp_cols / BCOLS; ++c) {
        const int col = col0 + c * BCOLS, cols = min(BCOLS, args.N - col);
        const bool in = c < blocks && ok;
        const uint32_t b = bufs == 1 ? 0 : tma_res ? reads & 1 : c & 1;
        uint8_t* yb = blk + b * TL::BLOCK_BYTES;
        uint8_t* pb = blk + TL::BLOCK_BYTES;
        OUT* yp = static_cast<OUT*>(args.C) + row0 * args.ldc + col;
        OUT* pp = static_cast<OUT*>(args.pre) + row0 * args.N + col;
        if (in && tma_res) {
          const uint32_t parity = bufs == 1 ? reads & 1u : (reads >> 1) & 1u;
          const bool here = mbar_wait_bounded(smem_u32(&bars[b]), parity, abort_flag, args.status, kWaitLimitNs);
          ok = __all_sync(0xffffffffu, here);
          if (ok) ++reads;
        } else if (in && res) {
          load_block<OUT>(static_cast<const OUT*>(args.residual) + row0 * args.ldr + col, args.ldr, rows, cols, lane, yb);
          __syncwarp();
        }
#pragma unroll 1
        for (int h = 0; h < PER; ++h) {
          const int at = (PER * c + h) * CW;   // first column of the warp's
          uint32_t v[CW];
          if constexpr (CW == 16) tmem_ld16(taddr + at, v); else tmem_ld32(taddr + at, v);
          if (at + CW == warp_cols) release_fill();   // the last read of the buffer
          float z[CW];
#pragma unroll
          for (int e = 0; e < CW; ++e) z[e] = __uint_as_float(v[e]);
          if (args.bias != nullptr) {
            float mine = bias[0];
#pragma unroll
            for (int k = 1; k < WARP_COLS / 32; ++k) mine = at / 32 == k ? bias[k] : mine;
#pragma unroll
            for (int e = 0; e < CW; ++e) z[e] += __shfl_sync(0xffffffffu, mine, at % 32 + e);
          }
          uint32_t w[16];
          if (args.pre != nullptr) {
            Row64<OUT>::pack(z, w);
            if constexpr (STAGED) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *block_piece<OUT>(pb, lane, 4 * h + j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            } else if (in && lane < rows) {
              store64(pp + lane * static_cast<int64_t>(args.N), args.al_pre, cols / 8, w);
            }
          }
          if constexpr (ACT == kActAny) {
            activate(z, args.act);
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e) z[e] = act_value<ACT>(z[e]);
          }
          if (res) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 u = *block_piece<OUT>(yb, lane, 4 * h + j);
              w[4 * j] = u.x;
              w[4 * j + 1] = u.y;
              w[4 * j + 2] = u.z;
              w[4 * j + 3] = u.w;
            }
            Row64<OUT>::add(z, w);
          }
          Row64<OUT>::pack(z, w);
          if constexpr (STAGED) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *block_piece<OUT>(yb, lane, 4 * h + j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          } else if (in && ok && lane < rows) {
            store64(yp + lane * args.ldc, args.al_c, cols / 8, w);
          }
        }
        if constexpr (STAGED) {
          __syncwarp();
          if (in && ok) {
            store_block<OUT, ALIGNED>(yp, args.ldc, args.al_c, rows, cols, lane, yb);
            if (args.pre != nullptr) store_block<OUT, ALIGNED>(pp, args.N, args.al_pre, rows, cols, lane, pb);
          }
        }
        // The buffer's next TMA load must not overtake these accesses, which can wait behind stores.
        if (tma_res) fence_proxy_async_smem();
        __syncwarp();
        if (in && tma_res && ok) load_residual(c + bufs);
      }
    }
    if (lane == 0)   // blocks still on their way after a failed wait
      for (; reads != loads; ++reads)
        mbar_wait_bounded(smem_u32(&bars[bufs == 1 ? 0 : reads & 1]), bufs == 1 ? reads & 1u : (reads >> 1) & 1u, never,
                          nullptr, kDrainLimitNs);
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // no CTA leaves while its partner may still use its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TL::TMEM_COLS);
  }
}

// What becomes of the `rest` tiles of a partial round, of `stages` pairs of K blocks (about half a
// microsecond) each: cut into `parts` along K, or narrow where that is allowed, or neither; and
// about the stages that the round then takes.  Joining s parts costs about as much as
// kJoin + kJoinPart s stages (they pass through scratch memory).
constexpr int kJoin = 12, kJoinPart = 4, kMaxParts = 8;
struct Rest {
  int parts;
  bool narrow;
  int64_t stages;
};
Rest plan_rest(int64_t rest, int64_t pairs, int64_t stages, bool narrow) {
  Rest best{1, false, rest > 0 ? stages : 0};
  if (rest == 0) return best;
  if (narrow && 2 * rest <= pairs) best = Rest{1, true, (3 * stages + 3) / 4};
  for (int s = 2; s <= kMaxParts && rest * s <= pairs && 2 * s <= stages; ++s) {
    const int64_t cost = (stages + s - 1) / s + kJoin + kJoinPart * s;
    if (cost < best.stages) best = Rest{s, false, cost};
  }
  return best;
}
// Of an M x N output in tiles of 256 x BN, in rounds of `pairs`.
template <int BN>
Rest plan_output(int64_t M, int64_t N, int64_t K, int64_t pairs, bool narrow) {
  const int64_t tiles = (M + BM - 1) / BM * ((N + BN - 1) / BN);
  return plan_rest(tiles % pairs, pairs, ((K + BK - 1) / BK + 1) / 2, narrow);
}
int64_t most_pairs(int sms) { return std::min(kMaxPairs, std::max(1, sms / 2)); }

// Bytes (32, 16 or 0 for less) that rows ld elements apart are aligned to.
int32_t row_alignment(const void* p, int64_t ld, size_t elem) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * elem);
  return v % 32 == 0 ? 32 : v % 16 == 0 ? 16 : 0;
}

template <int BN, bool A_MN, bool B_MN, typename OUT, int ACT, bool ALIGNED, bool NARROW = false>
cudaError_t launch_kernel(const LinearGemm& g, const Rest& plan, cudaStream_t s) {
  using TL = Tile<BN, sizeof(OUT) == 4>;
  Args a{};
  a.M = static_cast<int32_t>(g.M);
  a.N = g.N;
  a.K = g.K;
  a.m_tiles = static_cast<int32_t>((g.M + BM - 1) / BM);
  a.n_tiles = (g.N + BN - 1) / BN;
  a.bias = g.bias;
  a.residual = g.residual;
  a.pre = g.pre;
  a.C = g.C;
  a.ldr = g.ldr;
  a.ldc = g.ldc;
  a.status = g.status;
  a.act = g.act;
  a.part = g.part;
  a.db = g.db;
  a.db_parts = g.parts;
  a.db_cols = g.part_cols;
  a.al_c = row_alignment(g.C, g.ldc, sizeof(OUT));
  a.al_pre = row_alignment(g.pre, g.N, sizeof(OUT));
  CUtensorMap mA, mB;
  const uint64_t M = static_cast<uint64_t>(g.M), N = g.N, K = g.K;
  if (!(A_MN ? make_strided_map(&mA, MOE_BF16, g.A, M, K, g.lda, 64, BK)
             : make_strided_map(&mA, MOE_BF16, g.A, K, M, g.lda, BK, HALF)) ||
      !(B_MN ? make_strided_map(&mB, MOE_BF16, g.B, N, K, g.ldb, 64, BK)
             : make_strided_map(&mB, MOE_BF16, g.B, K, N, g.ldb, BK, TL::COLS)))
    return cudaErrorInvalidValue;
  CUtensorMap mR = mA, mBn = mB;
  if (NARROW && !make_strided_map(&mBn, MOE_BF16, g.B, K, N, g.ldb, BK, TL::COLS / 2)) return cudaErrorInvalidValue;
  if (ALIGNED && g.residual &&
      !make_strided_map(&mR, sizeof(OUT) == 4 ? MOE_F32 : MOE_BF16, g.residual, N, M, g.ldr, 32, 32, TL::ROW_BYTES))
    return cudaErrorInvalidValue;
  auto kern = linear_pair_kernel<BN, A_MN, B_MN, OUT, ACT, ALIGNED, NARROW>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), TL::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
  const int64_t most = most_pairs(device_sm_count()), rest = tiles % most;
  int64_t pairs = std::min(tiles, most);
  a.scratch = g.scratch;
  a.tickets = g.tickets;
  a.parts = plan.parts;
  a.whole = tiles;
  if (plan.parts > 1) {
    a.cut_tiles = static_cast<int32_t>(rest);
    pairs = tiles > rest ? most : rest * plan.parts;
  } else if (NARROW) {
    a.whole = tiles - rest;
    pairs = tiles > rest ? most : 2 * rest;
  }
  return launch_overlapped(kern, 2 * pairs, THREADS, TL::SMEM, s, 0, mA, mB, mBn, mR, a);
}

}  // namespace

namespace {

template <bool A_MN, bool B_MN, typename OUT, int ACT>
cudaError_t launch_typed(const LinearGemm& g, cudaStream_t s) {
  const size_t e = sizeof(OUT);
  const bool aligned = row_alignment(g.C, g.ldc, e) != 0 && (!g.pre || row_alignment(g.pre, g.N, e) != 0) &&
                       (!g.residual || row_alignment(g.residual, g.ldr, e) != 0) && g.N * e % 16 == 0;
  constexpr bool NARROWABLE = !B_MN && sizeof(OUT) == 2;
  const int64_t pairs = most_pairs(device_sm_count());
  // Gradients whose narrow tiles fit one round take those: half the columns are half the epilogue
  // and half the products of a pair, and with few pairs L2 keeps up (300 x 1024 x 1024: dx 11.9 -> 10.3
  // us; 300 x 1001 x 1000, unaligned: both gradients 35 -> 31 us; beyond one round 4096 x 2560 x 1280: 26 ->
  // 34 us).
  if constexpr (B_MN) {
    if ((g.M + BM - 1) / BM * ((g.N + 127) / 128) <= pairs) {
      const Rest plan = plan_output<128>(g.M, g.N, g.K, pairs, false);
      return aligned ? launch_kernel<128, A_MN, B_MN, OUT, ACT, true>(g, plan, s)
                     : launch_kernel<128, A_MN, B_MN, OUT, kActAny, false>(g, plan, s);
    }
  }
  const Rest plan = plan_output<256>(g.M, g.N, g.K, pairs, NARROWABLE);
  if constexpr (NARROWABLE) {
    if (plan.narrow)
      return aligned ? launch_kernel<256, A_MN, B_MN, OUT, ACT, true, true>(g, plan, s)
                     : launch_kernel<256, A_MN, B_MN, OUT, kActAny, false, true>(g, plan, s);
  }
  return aligned ? launch_kernel<256, A_MN, B_MN, OUT, ACT, true>(g, plan, s)
                 : launch_kernel<256, A_MN, B_MN, OUT, kActAny, false>(g, plan, s);
}

template <typename OUT>
cudaError_t launch_forward(const LinearGemm& g, cudaStream_t s) {
#define MOE_CALL(ACT) launch_typed<false, false, OUT, ACT>(g, s)
  MOE_DISPATCH_ACT(g.act, MOE_CALL)
#undef MOE_CALL
}

}  // namespace

int64_t pair_cycles(int64_t M, int64_t N, int64_t K, bool f32, int sms) {
  const int64_t tiles = (M + BM - 1) / BM * ((N + 255) / 256), pairs = most_pairs(sms);
  const int64_t stages = ((K + BK - 1) / BK + 1) / 2, last = plan_output<256>(M, N, K, pairs, !f32).stages;
  return 20000 + (tiles / pairs * stages + last) * 2 * (tiles <= pairs ? 640 : 573);
}

// About 0.2 us per sum and lane, beside rounds of about half a microsecond per stage; the few stages
// that a cut leaves, and what a launch takes, are in the constants.
bool pair_hides_sums(const LinearGemm& g, int sms) {
  const int64_t tiles = (g.M + BM - 1) / BM * ((g.N + 255) / 256), pairs = most_pairs(sms);
  const int64_t stages = (g.K + 2 * BK - 1) / (2 * BK), rounds = (tiles + pairs - 1) / pairs;
  return g.part_cols * g.parts <= 128 * std::min(tiles, pairs) * (16 + stages * rounds / 4);
}

cudaError_t launch_linear_pair(const LinearGemm& g, cudaStream_t s) {
  const bool f32 = g.out_dtype == MOE_F32;
  if (g.a_mn)
    return f32 ? launch_typed<true, true, float, MOE_ACT_NONE>(g, s)
               : launch_typed<true, true, __nv_bfloat16, MOE_ACT_NONE>(g, s);
  if (g.b_mn)
    return f32 ? launch_typed<false, true, float, MOE_ACT_NONE>(g, s)
               : launch_typed<false, true, __nv_bfloat16, MOE_ACT_NONE>(g, s);
  return f32 ? launch_forward<float>(g, s) : launch_forward<__nv_bfloat16>(g, s);
}

}  // namespace moe
