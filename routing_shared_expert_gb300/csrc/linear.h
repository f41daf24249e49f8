// Internal declarations of the dense projection's matrix products.
#pragma once

#include "internal.h"
#include "launch.h"

namespace moe {

// C[m][n] = epilogue(sum_k A(m, k) B(n, k)): A and B bf16 with 16-byte aligned rows, either
// K-major (a row per m or n, K contiguous) or MN-major (a row per k, M or N contiguous).
//   z = sum + bias[n];  pre[m][n] = z;  C[m][n] = act(z) + residual[m][n]
struct LinearGemm {
  const void* A;
  const void* B;
  int64_t lda, ldb;        // elements between rows
  bool a_mn, b_mn;
  int64_t M;
  int32_t N, K;
  int32_t out_dtype;       // of C, pre and residual
  int32_t act;
  const float* bias;       // [N] or nullptr
  const void* residual;    // [M][ldr] or nullptr
  void* pre;               // [M][N] or nullptr
  void* C;                 // [M][ldc]
  int64_t ldr, ldc;
  int32_t* status;
  float* scratch;          // kPairScratchFloats: partial tiles of launch_linear_pair
  unsigned* tickets;       // kPairTicketBytes, zero between calls
  // Gradients: db[c] = sum of part[b][c] over b < parts, for c < part_cols, beside the products (db
  // nullptr: none).
  const float* part;
  int64_t parts;
  int32_t part_cols;
  float* db;
};

// Most CTA pairs of a launch, and the partial tiles (256 x 256 per pair) and arrival counts (a
// byte per cut tile and CTA of the pair) its cut tiles need.
constexpr int kMaxPairs = 76;
constexpr size_t kPairScratchFloats = static_cast<size_t>(kMaxPairs) * 256 * 256;
constexpr size_t kPairTicketOffset = 64;   // bytes into the workspace header
constexpr size_t kPairTicketBytes = 2 * kMaxPairs;
static_assert(kPairTicketOffset + kPairTicketBytes <= 256, "the counts lie in the header");

// CTA pairs, 256 x 256 tiles (gemm_linear.cu).
cudaError_t launch_linear_pair(const LinearGemm& g, cudaStream_t s);
// About the cycles of a launch_linear_pair: its rounds of tiles (a K block takes 573 cycles once
// the operands are in L2, 640 in a single round), or of their parts, and what a launch costs.  f32:
// the output's type.
int64_t pair_cycles(int64_t M, int64_t N, int64_t K, bool f32, int sms);
// Whether such a launch hides those sums: each of its lanes adds few enough of them.
bool pair_hides_sums(const LinearGemm& g, int sms);
// One to kVecTokens rows of A (both operands K-major, any alignment), a warp per row of B
// (linear_vec.cu).
constexpr int kVecTokens = 4;
cudaError_t launch_linear_vec(const LinearGemm& g, cudaStream_t s);
// Few rows of A (both operands K-major), depth split over a cluster (gemm_linear_few.cu).
cudaError_t launch_linear_few(const LinearGemm& g, cudaStream_t s);
struct FewShape {
  int tokens;        // per tile
  int split;         // CTAs per cluster
  bool one_round;    // every tile has a CTA resident at once
  int64_t cycles;    // about what the launch takes
};
FewShape few_shape(int64_t T, int64_t N, int64_t K, int sms);

}  // namespace moe
