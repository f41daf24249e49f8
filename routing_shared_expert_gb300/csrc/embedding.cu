// Token embedding: out_t = scale table[id_t], and the gradient of the table by tokens,
// dtable_v = scale sum_{t: id_t = v} dout_t, summed in fp32 in a fixed order.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

struct EmbedArgs {
  const void* ids;
  const void* src;       // table, or dout
  void* dst;             // out, or dtable
  int64_t T, V, ldt, ldo;
  int32_t d, accumulate;
  float scale;
  int32_t* status;
};

// The token's row, -1 for none; a number outside the table is reported by the callers that pass a
// status word.
template <typename I>
__device__ __forceinline__ int64_t token_row(const I* ids, int64_t t, int64_t V, int32_t* status) {
  const int64_t v = ids[t];
  if (v >= 0 && v < V) return v;
  if (v != -1) set_status(status, MOE_ERR_DEVICE_BOUNDS);
  return -1;
}

template <typename I, typename W, typename Y>
__global__ void __launch_bounds__(128) embed_any_kernel(EmbedArgs a) {
  const int64_t t = blockIdx.x;
  const int64_t v = token_row(static_cast<const I*>(a.ids), t, a.V, a.status);
  Y* out = static_cast<Y*>(a.dst) + t * a.ldo;
  const W* row = static_cast<const W*>(a.src) + (v < 0 ? 0 : v) * a.ldt;
  for (int c = threadIdx.x; c < a.d; c += blockDim.x)
    out[c] = from_f32<Y>(v < 0 ? 0.f : to_f32(row[c]) * a.scale);
}

// Gradient without a sort: a CTA owns kScanRows rows of the table and 256 columns, reads every
// token number, keeps those of its rows in order, and adds their gradients up in shared memory,
// a thread per column.
constexpr int kScanRows = 32, kScanIds = 8 * 256;

template <typename I, typename Y, typename W>
__global__ void __launch_bounds__(256) embed_scan_kernel(EmbedArgs a) {
  __shared__ float acc[kScanRows][256];
  __shared__ int32_t list_t[kScanIds];
  __shared__ uint8_t list_v[kScanIds];
  __shared__ int32_t warp_n[8];
  __shared__ uint32_t seen;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kScanRows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + tid;
  int32_t* status = blockIdx.x == 0 && blockIdx.y == 0 ? a.status : nullptr;
  for (int r = 0; r < kScanRows; ++r) acc[r][tid] = 0.f;
  if (tid == 0) seen = 0;
  for (int64_t t0 = 0; t0 < a.T; t0 += kScanIds) {
    // eight neighbouring tokens per thread, so that the list is in the tokens' order
    uint32_t hits = 0;
    int row[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + tid * 8 + j;
      const int64_t v = t < a.T ? token_row(static_cast<const I*>(a.ids), t, a.V, status) : -1;
      row[j] = static_cast<int>(v - v0);
      if (v >= v0 && v < v0 + kScanRows) hits |= 1u << j;
    }
    int n = __popc(hits), before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    __syncthreads();   // the last tile's list and counts are used up
    if (lane == 31) warp_n[warp] = before;
    __syncthreads();
    int at = before - n, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += warp_n[w];
      total += warp_n[w];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (hits >> j & 1) {
        list_t[at] = static_cast<int32_t>(t0 + tid * 8 + j);
        list_v[at++] = static_cast<uint8_t>(row[j]);
        atomicOr(&seen, 1u << row[j]);
      }
    __syncthreads();
    if (c < a.d)
      for (int i = 0; i < total; ++i)
        acc[list_v[i]][tid] += to_f32(static_cast<const Y*>(a.src)[list_t[i] * a.ldo + c]);
  }
  __syncthreads();
  if (c >= a.d) return;
  for (int r = 0; r < kScanRows && v0 + r < a.V; ++r) {
    W* out = static_cast<W*>(a.dst) + (v0 + r) * a.ldt + c;
    const float v = acc[r][tid] * a.scale;
    if (!a.accumulate) *out = from_f32<W>(v);
    else if (seen >> r & 1) *out = from_f32<W>(to_f32(*out) + v);
  }
}

// ---------------------------------------------------------------------- launch --

template <typename I, typename W, typename Y>
cudaError_t launch_embed(const EmbedArgs& a, bool backward, cudaStream_t s) {
  if (!backward) {
    embed_any_kernel<I, W, Y><<<static_cast<unsigned>(a.T), 128, 0, s>>>(a);
  } else {
    const dim3 grid(static_cast<unsigned>((a.V + kScanRows - 1) / kScanRows), static_cast<unsigned>((a.d + 255) / 256));
    embed_scan_kernel<I, Y, W><<<grid, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}
template <typename I, typename W>
cudaError_t launch_embed_out(const EmbedArgs& a, const moe_embedding_config& c, bool backward, cudaStream_t s) {
  return c.out_dtype == MOE_F32 ? launch_embed<I, W, float>(a, backward, s)
                                : launch_embed<I, W, __nv_bfloat16>(a, backward, s);
}
template <typename I>
cudaError_t launch_embed_table(const EmbedArgs& a, const moe_embedding_config& c, bool backward, cudaStream_t s) {
  return c.table_dtype == MOE_F32 ? launch_embed_out<I, float>(a, c, backward, s)
                                  : launch_embed_out<I, __nv_bfloat16>(a, c, backward, s);
}

// ---------------------------------------------------------------------- checks --

constexpr int64_t kMaxTokens = int64_t{1} << 26, kMaxVocab = int64_t{1} << 30, kMaxElements = int64_t{1} << 40;
constexpr int32_t kMaxWidth = 1 << 20;

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
uintptr_t size_of(int32_t t) { return t == MOE_F32 ? 4 : 2; }
bool embed_sizes_ok(int64_t T, int64_t V, int32_t d) {
  return T >= 0 && T <= kMaxTokens && V >= 1 && V <= kMaxVocab && d >= 1 && d <= kMaxWidth;
}
size_t embed_workspace(int64_t, int64_t, int32_t) { return 256; }

moe_status run_embed(const moe_embedding_config* c, const void* ids, const void* src, void* dst,
                     bool backward, int32_t accumulate, void* workspace, size_t bytes, cudaStream_t s) {
  if (!c || !embed_sizes_ok(c->T, c->V, c->d) || !std::isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(c->table_dtype) || !dtype_ok(c->out_dtype) || (c->ids_int64 != 0 && c->ids_int64 != 1) ||
      (accumulate != 0 && accumulate != 1))
    return MOE_ERR_INVALID_ARG;
  const int64_t ldt = c->V > 1 && c->ldt ? c->ldt : c->d, ldo = c->T > 1 && c->ldo ? c->ldo : c->d;
  if (ldt < c->d || ldo < c->d) return MOE_ERR_INVALID_ARG;
  if (ldt > kMaxElements / c->V || (c->T > 0 && ldo > kMaxElements / c->T)) return MOE_ERR_UNSUPPORTED;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  const bool table = !backward || c->T > 0 || !accumulate;   // whether the table is looked at
  if (c->T == 0 && !backward) return MOE_OK;
  if (c->T > 0 && (!ids || !(backward ? src : dst))) return MOE_ERR_INVALID_ARG;
  if (table && !(backward ? dst : src)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(ids, c->ids_int64 ? 8 : 4) || !aligned_to(src, size_of(backward ? c->out_dtype : c->table_dtype)) ||
      !aligned_to(dst, size_of(backward ? c->table_dtype : c->out_dtype)) || !aligned_to(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (bytes < embed_workspace(c->T, c->V, c->d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (c->T == 0 && accumulate) return MOE_OK;
  EmbedArgs a{};
  a.ids = ids;
  a.src = src;
  a.dst = dst;
  a.T = c->T;
  a.V = c->V;
  a.ldt = ldt;
  a.ldo = ldo;
  a.d = c->d;
  a.accumulate = accumulate;
  a.scale = c->scale;
  a.status = static_cast<int32_t*>(workspace);
  const cudaError_t e = c->ids_int64 ? launch_embed_table<int64_t>(a, *c, backward, s)
                                     : launch_embed_table<int32_t>(a, *c, backward, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_embedding_workspace_size(int64_t T, int64_t V, int32_t d, size_t* bytes) {
  if (!bytes || !moe::embed_sizes_ok(T, V, d)) return MOE_ERR_INVALID_ARG;
  *bytes = moe::embed_workspace(T, V, d);
  return MOE_OK;
}

moe_status moe_embedding_forward(const moe_embedding_config* cfg, const void* ids, const void* table,
                                 void* out, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
  return moe::run_embed(cfg, ids, table, out, false, 0, workspace, workspace_bytes, stream);
}

moe_status moe_embedding_backward(const moe_embedding_config* cfg, const void* ids, const void* dout,
                                  void* dtable, int32_t accumulate, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  return moe::run_embed(cfg, ids, dout, dtable, true, accumulate, workspace, workspace_bytes, stream);
}

}  // extern "C"
