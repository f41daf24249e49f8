// Token embedding: the lookup, and the checks and entry points of both passes.
//
//   out_t = scale table[id_t],   dtable_v = scale sum_{t: id_t = v} dout_t
#include "embedding.cuh"

namespace moe {
namespace {

// Eight values that nothing reads soon: first to leave L2, where the rows of frequent tokens stay (131072 x 2560 in
// bf16 128.5 -> 125.7 us).
__device__ __forceinline__ void store8_once(__nv_bfloat16* p, const float2 (&v)[4]) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(pack_bf16x2(v[0].x, v[0].y)),
               "r"(pack_bf16x2(v[1].x, v[1].y)), "r"(pack_bf16x2(v[2].x, v[2].y)), "r"(pack_bf16x2(v[3].x, v[3].y))
               : "memory");
}
__device__ __forceinline__ void store8_once(float* p, const float2 (&v)[4]) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0].x), "f"(v[0].y),
               "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
               : "memory");
}

// A warp per token and slice of kSlice columns, its four loads of eight values per lane on their way at
// once; of rows of at most 256 columns (SHORT) the four loads, and a row's unused lanes where rows are aligned, go to
// further tokens.  ALIGNED: rows of the table and of out begin on groups of eight and end on one; else the groups are
// those of out, and the table's values are moved into place.
// Bound by HBM where rows are long: 131072 x 2560 fp32 -> bf16 157 us, 6.2 TB/s of DRAM traffic (a third of the rows that
// come again have left L2 by then, 120 MB of reading more); 24 tokens of 4096: 1.6 us, the latency of two reads.
constexpr int kSlice = 1024;

template <typename I, typename W, typename Y, bool ALIGNED, bool SHORT>
__global__ void __launch_bounds__(256) embed_kernel(EmbedArgs a, int slices, int64_t items) {
  launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (item >= items) return;
  const int lane = threadIdx.x & 31;
  const float2 scale = both(a.scale);
  wait_for_previous();
  if (ALIGNED) {
    // load k: columns from c on of token t[k].  SHORT: `slices` tokens to a warp's width
    const int lanes = SHORT ? 32 / slices : 32;
    const int64_t t0 = SHORT ? item * (4 * slices) + lane / lanes : item / slices;
    const int c0 = SHORT ? 8 * (lane & (lanes - 1)) : static_cast<int>(item - t0 * slices) * kSlice + 8 * lane;
    int64_t v[4];
#pragma unroll
    for (int k = 0; k < (SHORT ? 4 : 1); ++k) {
      const int64_t t = t0 + k * slices;
      v[k] = !SHORT || t < a.T ? token_row(static_cast<const I*>(a.ids), t, a.V, c0 == 0 ? a.status : nullptr) : -1;
    }
    uint32_t w[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t row = v[SHORT ? k : 0];
      const int c = SHORT ? c0 : c0 + 256 * k;
      if (c < a.d && row >= 0) load8(static_cast<const W*>(a.src) + row * a.ldt + c, w[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = SHORT ? t0 + k * slices : t0;
      const int c = SHORT ? c0 : c0 + 256 * k;
      if (c >= a.d || (SHORT && t >= a.T)) break;
      float2 u[4];
      unpack8<W>(w[k], u);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = v[SHORT ? k : 0] < 0 ? both(0.f) : mul2(u[j], scale);
      store8_once(static_cast<Y*>(a.dst) + t * a.ldo + c, u);
    }
  } else if (SHORT) {
    Slice<W, false> w[4];
    int64_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = item * 4 + k;
      v[k] = t < a.T ? token_row(static_cast<const I*>(a.ids), t, a.V, lane == 0 ? a.status : nullptr) : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v[k] >= 0) w[k].load(static_cast<const W*>(a.src) + v[k] * a.ldt, 0, a.d);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (item * 4 + k >= a.T) break;
      float2 u[4];
      w[k].unpack(u);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = v[k] < 0 ? both(0.f) : mul2(u[j], scale);
      store_slice<Y, false>(static_cast<Y*>(a.dst) + (item * 4 + k) * a.ldo, 0, a.d, u);
    }
  } else {
    const int64_t t = item / slices;
    const int c0 = static_cast<int>(item - t * slices) * kSlice;
    const int64_t v = token_row(static_cast<const I*>(a.ids), t, a.V, lane == 0 ? a.status : nullptr);
    Y* out = static_cast<Y*>(a.dst) + t * a.ldo;
    const W* row = static_cast<const W*>(a.src) + (v < 0 ? 0 : v) * a.ldt;
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(out) / sizeof(Y)) & 7;
    const Span span = span_of(a.src, a.V, a.ldt, a.d, sizeof(W));
    // the last slice takes the groups that the phase pushes past its end
    const int end = c0 + kSlice >= a.d ? a.d + phase : c0 + kSlice;
    for (int g = c0 + 8 * lane; g < end; g += 256) {
      const int e0 = g - phase;
      float2 u[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
      if (v >= 0) take_any(row + e0, e0, a.d, span, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], scale);
      if (e0 >= 0 && e0 + 8 <= a.d) {
        store8(out + e0, u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j >= 0 && e0 + j < a.d) out[e0 + j] = from_f32<Y>(j & 1 ? u[j / 2].y : u[j / 2].x);
      }
    }
  }
}

// ---------------------------------------------------------------------- launch --

template <typename I, typename W, typename Y>
cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t s) {
  const bool aligned = groups_of_eight<W>(a.src, a.ldt, a.d) && groups_of_eight<Y>(a.dst, a.ldo, a.d);
  // several tokens to a warp where there are warps enough for all SMs
  if (a.d <= kColumns && a.T >= 4096) {
    int lanes = 32;
    while (aligned && 8 * (lanes / 2) >= a.d) lanes /= 2;
    const int tokens = 32 / lanes;
    const int64_t items = (a.T + 4 * tokens - 1) / (4 * tokens);
    const dim3 grid(static_cast<unsigned>((items + 7) / 8));
    return aligned ? launch_over(embed_kernel<I, W, Y, true, true>, grid, 256, 0, s, a, tokens, items)
                   : launch_over(embed_kernel<I, W, Y, false, true>, grid, 256, 0, s, a, 1, items);
  }
  const int slices = (a.d + kSlice - 1) / kSlice;
  const int64_t items = a.T * slices;
  const dim3 grid(static_cast<unsigned>((items + 7) / 8));
  return aligned ? launch_over(embed_kernel<I, W, Y, true, false>, grid, 256, 0, s, a, slices, items)
                 : launch_over(embed_kernel<I, W, Y, false, false>, grid, 256, 0, s, a, slices, items);
}
template <typename I, typename W>
cudaError_t launch_out(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.out_dtype == MOE_F32 ? launch_embed<I, W, float>(a, s) : launch_embed<I, W, __nv_bfloat16>(a, s);
}
template <typename I>
cudaError_t launch_table(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.table_dtype == MOE_F32 ? launch_out<I, float>(a, c, s) : launch_out<I, __nv_bfloat16>(a, c, s);
}
cudaError_t launch_forward(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.ids_int64 ? launch_table<int64_t>(a, c, s) : launch_table<int32_t>(a, c, s);
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
size_t embed_workspace(int64_t T, int64_t V, int32_t d) { return 256 + embedding_scratch(T, V, d); }

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
  if (bytes < (backward ? embed_workspace(c->T, c->V, c->d) : 256)) return MOE_ERR_WORKSPACE_TOO_SMALL;
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
  a.scratch = static_cast<char*>(workspace) + 256;
  const cudaError_t e = backward ? launch_embedding_backward(a, *c, s) : launch_forward(a, *c, s);
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
