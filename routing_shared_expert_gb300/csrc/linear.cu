// Dense projections of the block: y = act(x W^T + b) + r and the gradients dx, dW, db.
//
//   z = x W^T + b,  y = act(z) + r
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_t dz
//
// The products run on the tensor cores (gemm_linear.cu; gemm_linear_few.cu for few tokens).
// Here: the argument checks, the pass that forms dz (rounded to bf16, which the products need,
// while db sums the unrounded values) and the copy that gives unaligned operands 16-byte rows.
#include "linear.h"
#include "load_any.cuh"

#include <algorithm>

#include "activation.cuh"

namespace moe {
namespace {

constexpr int kDzRows = 64;     // rows per block of the dz pass, and per partial sum of db
constexpr int kDzCols = 256;    // columns per block: 8 per lane

// Which kernel takes a forward product.  A warp per weight row (linear_vec.cu) needs no aligned
// copies and starts soonest, but reads x anew for every row: it wins for one token up to about
// 2^25 weights (2048 x 2048: 5.0 us against 6.0; 7168 x 7168: 20.3 against 20.0) and for up to
// four where the whole product is small (512 x 512: 2.7 against 4.3; two tokens of 2048 x 2048:
// 6.8 against 6.5).  Unaligned rows spare it the copies: one token of 4095 x 14336 46.8 against
// 63.7, two of 2047 x 2047 9.4 against 10.3, of 2810 x 2816 17.1 against 13.7.
// The few-token kernel wins while its tiles are resident at once and its loads take less than
// the pair kernel's rounds (384 tokens of 2048 x 5632: 17.1 us against 19.2; 512: 29.7
// against 19.6).
enum class Form { kVec, kFew, kPair };
Form forward_form(int64_t T, int64_t N, int64_t K, bool f32, bool aligned) {
  const int64_t most = T == 1 ? int64_t{1} << 25 : T == 2 && !aligned ? int64_t{1} << 23 : int64_t{1} << 22;
  if (T <= kVecTokens && (T * N * K <= most || (T == 1 && !aligned))) return Form::kVec;
  const int sms = device_sm_count();
  const FewShape f = few_shape(T, N, K, sms);
  return f.one_round && f.cycles < pair_cycles(T, N, K, f32, sms) ? Form::kFew : Form::kPair;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

struct DzArgs {
  const void* dy;
  const void* pre;              // nullptr: the identity
  int64_t ldy, T, col_blocks, ld_dz;
  int32_t n;
  __nv_bfloat16* dz;            // [T][ld_dz] or nullptr
  float* part;                  // [row blocks][n] or nullptr
};

// dz = dy act'(pre) and, per block of kDzRows rows, its column sums (each warp its rows in
// order, then the warps in order).  VEC: 16-byte loads of whole groups of eight columns.
//
// dz is rounded to bf16 whatever the types of dy, dx and dW: a product on the tensor cores takes both
// operands in one 16-bit type, and the others, x and W, are bf16.  With bf16 results the error of dx and
// dW is 2.35e-3 (rms, relative) against 1.66e-3 if only they were rounded; with fp32 ones it is 1.7e-3.
// The rest dz - bf16(dz) as a second operand would bring that to a few 10^-6 and take dx and dW twice
// as long.
template <typename OUT, bool VEC, int ACT>
__global__ void __launch_bounds__(256) dz_kernel(DzArgs a) {
  __shared__ float s_sum[8][kDzCols];
  launch_dependents();
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t rb = blockIdx.x / a.col_blocks;
  const int c0 = static_cast<int>(blockIdx.x % a.col_blocks) * kDzCols + lane * 8;
  const int64_t t1 = min(a.T, (rb + 1) * kDzRows);
  float sum[8] = {};
  if (c0 < a.n) {
    const Span sy = span_of(a.dy, a.T, a.ldy, a.n, sizeof(OUT)), sp = span_of(a.pre, a.T, a.n, a.n, sizeof(OUT));
    for (int64_t t = rb * kDzRows + warp; t < t1; t += 8) {
      const OUT* dy = static_cast<const OUT*>(a.dy) + t * a.ldy + c0;
      const OUT* pre = static_cast<const OUT*>(a.pre) + t * a.n + c0;
      float g[8], z[8];
      if (VEC) {
        load8(dy, g);
        if (ACT != MOE_ACT_NONE) load8(pre, z);
      } else {
        const Raw8 rg = load8_raw(dy, sy);
        Raw8 rz;
        if (ACT != MOE_ACT_NONE) rz = load8_raw(pre, sp);
        take8(rg, dy, a.n - c0, g);
        if (ACT != MOE_ACT_NONE) take8(rz, pre, a.n - c0, z);
      }
      if (ACT != MOE_ACT_NONE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= act_slope<ACT>(z[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
      if (a.dz)   // ld_dz is a multiple of 8: whole groups, the last one padded
        *reinterpret_cast<uint4*>(a.dz + t * a.ld_dz + c0) =
            make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                       pack_bf16x2(g[6], g[7]));
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) s_sum[warp][lane * 8 + e] = sum[e];
  __syncthreads();
  const int col = static_cast<int>(blockIdx.x % a.col_blocks) * kDzCols + threadIdx.x;
  if (col < a.n) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += s_sum[w][threadIdx.x];
    a.part[rb * a.n + col] = v;
  }
}

template <typename OUT, int ACT>
cudaError_t launch_dz_act(const DzArgs& a, bool vec, cudaStream_t s) {
  const int64_t grid = (a.T + kDzRows - 1) / kDzRows * a.col_blocks;
  return vec ? launch_overlapped(dz_kernel<OUT, true, ACT>, grid, 256, 0, s, 0, a)
             : launch_overlapped(dz_kernel<OUT, false, ACT>, grid, 256, 0, s, 0, a);
}
template <typename OUT>
cudaError_t launch_dz(const DzArgs& a, int act, bool vec, cudaStream_t s) {
#define MOE_CALL(ACT) launch_dz_act<OUT, ACT>(a, vec, s)
  MOE_DISPATCH_ACT(act, MOE_CALL)
#undef MOE_CALL
}

// db: 32 columns per CTA, 32 warps that each add every 32nd block, then the warps in order.
__global__ void __launch_bounds__(1024) db_kernel(const float* part, int64_t blocks, int n, float* db) {
  __shared__ float s_sum[32][33];
  launch_dependents();
  wait_for_previous();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (col < n)
    for (int64_t b = w; b < blocks; b += 32) sum += part[b * n + col];
  s_sum[w][lane] = sum;
  __syncthreads();
  if (w == 0 && col < n) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s_sum[i][lane];
    db[col] = v;
  }
}

// Rows of cols bf16 values, ld apart, to rows ldd (a multiple of 8) apart: eight values per
// thread and step, zeros past cols.
__global__ void __launch_bounds__(256) align_rows_kernel(const __nv_bfloat16* src, int64_t rows, int cols,
                                                         int64_t ld, __nv_bfloat16* dst, int64_t ldd) {
  launch_dependents();
  wait_for_previous();
  const int64_t per = ldd / 8, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * per; i += step) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i - r * per) * 8;
    const unsigned short* s = reinterpret_cast<const unsigned short*>(src + r * ld);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? s[c + e] : 0u;
    *reinterpret_cast<uint4*>(dst + r * ldd + c) =
        make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

int64_t up8(int64_t v) { return (v + 7) & ~int64_t{7}; }

// Elements between rows: dense ones for 0, and for a single row, whose stride may be anything.
int64_t row_stride(int64_t ld, int64_t rows, int32_t cols) { return ld == 0 || rows == 1 ? cols : ld; }

struct LinearLayout {
  size_t dz, db_part, x, w, scratch, total;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

LinearLayout linear_layout(const moe_linear_config& c) {
  LinearLayout L{};
  size_t o = 256;
  L.dz = o;
  o = up256(o + static_cast<size_t>(c.T) * up8(c.out_features) * 2);
  L.db_part = o;
  o = up256(o + static_cast<size_t>((c.T + kDzRows - 1) / kDzRows) * c.out_features * 4);
  L.x = o;      // aligned copies of x and W
  o = up256(o + static_cast<size_t>(c.T) * up8(c.in_features) * 2);
  L.w = o;
  o = up256(o + static_cast<size_t>(c.out_features) * up8(c.in_features) * 2);
  L.scratch = o;
  o = up256(o + kPairScratchFloats * 4);
  L.total = o;
  return L;
}

// The operand itself where its rows start on 16-byte boundaries, else an aligned copy.
struct Operand {
  const void* p;
  int64_t ld;
};
cudaError_t aligned_operand(const void* p, int64_t rows, int32_t cols, int64_t ld, void* copy, Operand* o,
                            cudaStream_t s) {
  if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld % 8 == 0 || rows == 1)) {
    *o = {p, up8(ld)};
    return cudaSuccess;
  }
  *o = {copy, up8(cols)};
  const int64_t blocks = std::min<int64_t>((rows * (o->ld / 8) + 255) / 256, static_cast<int64_t>(device_sm_count()) * 32);
  return launch_overlapped(align_rows_kernel, blocks, 256, 0, s, 0, static_cast<const __nv_bfloat16*>(p), rows, cols, ld,
                           static_cast<__nv_bfloat16*>(copy), o->ld);
}

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool elem_aligned(const void* p, int32_t t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == MOE_F32 ? 3u : 1u)) == 0;
}

moe_status check_linear(const moe_linear_config* c) {
  if (!c || c->T < 0 || c->T > (int64_t{1} << 28)) return MOE_ERR_INVALID_ARG;
  if (c->in_features < 1 || c->out_features < 1 || c->in_features > (1 << 20) || c->out_features > (1 << 20))
    return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(c->dtype) || !dtype_ok(c->out_dtype) || !dtype_ok(c->dx_dtype) || !dtype_ok(c->dw_dtype))
    return MOE_ERR_INVALID_ARG;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if ((c->ldx && c->ldx < c->in_features) || (c->ldw && c->ldw < c->in_features) ||
      (c->ldr && c->ldr < c->out_features) || (c->ldy && c->ldy < c->out_features))
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  // byte offsets within 2^46, and products of tile counts within 64 bits
  const int64_t most = int64_t{1} << 44;
  for (int64_t ld : {c->ldx, c->ldw, c->ldr, c->ldy})
    if (ld < 0 || ld > most / std::max<int64_t>(1, std::max<int64_t>(c->T, c->out_features)))
      return MOE_ERR_INVALID_ARG;
  if (c->T * std::max<int64_t>(c->in_features, c->out_features) > (int64_t{1} << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_linear_ws(const moe_linear_config& c, void* ws, size_t bytes) {
  if (!ws) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_MISALIGNED;
  return bytes < linear_layout(c).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_linear_workspace_size(const moe_linear_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_linear(cfg);
  if (s != MOE_OK) return s;
  *bytes = moe::linear_layout(*cfg).total;
  return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_config* cfg, const void* x, const void* W,
                              const float* bias, const void* residual, void* pre, void* y,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace moe;
  moe_status s = check_linear(cfg);
  if (s != MOE_OK) return s;
  const moe_linear_config& c = *cfg;
  if ((s = check_linear_ws(c, workspace, workspace_bytes)) != MOE_OK) return s;
  if (c.T == 0) return MOE_OK;
  if (!x || !W || !y) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, MOE_BF16) || !elem_aligned(W, MOE_BF16) || !elem_aligned(bias, MOE_F32) ||
      !elem_aligned(residual, c.out_dtype) || !elem_aligned(pre, c.out_dtype) ||
      !elem_aligned(y, c.out_dtype))
    return MOE_ERR_MISALIGNED;
  const LinearLayout L = linear_layout(c);
  char* ws = static_cast<char*>(workspace);
  const int64_t ldx = row_stride(c.ldx, c.T, c.in_features), ldw = row_stride(c.ldw, c.out_features, c.in_features);
  const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(W)) & 15u) == 0 &&
                       (ldx % 8 == 0 || c.T == 1) && ldw % 8 == 0;
  const Form form = forward_form(c.T, c.out_features, c.in_features, c.out_dtype == MOE_F32, aligned);
  Operand ox{x, ldx}, ow{W, ldw};
  if (form != Form::kVec && (aligned_operand(x, c.T, c.in_features, ldx, ws + L.x, &ox, stream) != cudaSuccess ||
               aligned_operand(W, c.out_features, c.in_features, ldw, ws + L.w, &ow, stream) != cudaSuccess))
    return MOE_ERR_CUDA;
  LinearGemm g{};
  g.A = ox.p;
  g.lda = ox.ld;
  g.B = ow.p;
  g.ldb = ow.ld;
  g.M = c.T;
  g.N = c.out_features;
  g.K = c.in_features;
  g.out_dtype = c.out_dtype;
  g.act = c.act;
  g.bias = bias;
  g.residual = residual;
  g.pre = pre;
  g.C = y;
  g.ldr = row_stride(c.ldr, c.T, c.out_features);
  g.ldc = row_stride(c.ldy, c.T, c.out_features);
  g.status = static_cast<int32_t*>(workspace);
  g.scratch = reinterpret_cast<float*>(ws + L.scratch);
  g.tickets = reinterpret_cast<unsigned*>(ws + kPairTicketOffset);
  const cudaError_t e = form == Form::kVec   ? launch_linear_vec(g, stream)
                        : form == Form::kFew ? launch_linear_few(g, stream)
                                             : launch_linear_pair(g, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_linear_backward(const moe_linear_config* cfg, const void* x, const void* W,
                               const void* pre, const void* dy, void* dx, void* dW, float* dbias,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace moe;
  moe_status s = check_linear(cfg);
  if (s != MOE_OK) return s;
  const moe_linear_config& c = *cfg;
  if ((s = check_linear_ws(c, workspace, workspace_bytes)) != MOE_OK) return s;
  if (!elem_aligned(x, MOE_BF16) || !elem_aligned(W, MOE_BF16) || !elem_aligned(pre, c.out_dtype) ||
      !elem_aligned(dy, c.out_dtype) || !elem_aligned(dx, c.dx_dtype) || !elem_aligned(dW, c.dw_dtype) ||
      !elem_aligned(dbias, MOE_F32))
    return MOE_ERR_MISALIGNED;
  if (c.T == 0) {
    const size_t n = static_cast<size_t>(c.out_features);
    if (dW && cudaMemsetAsync(dW, 0, n * c.in_features * (c.dw_dtype == MOE_F32 ? 4 : 2), stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, n * 4, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dy || (c.act != MOE_ACT_NONE && !pre) || (dW && !x) || (dx && !W)) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(c);
  char* ws = static_cast<char*>(workspace);
  const int64_t ldy = row_stride(c.ldy, c.T, c.out_features);
  const int32_t n = c.out_features;
  const int64_t blocks = (c.T + kDzRows - 1) / kDzRows;
  const bool identity = c.act == MOE_ACT_NONE;
  Operand oz{dy, ldy};
  // dy is dz where nothing has to be multiplied or rounded and its rows are aligned
  const bool as_is = identity && c.out_dtype == MOE_BF16 && (reinterpret_cast<uintptr_t>(dy) & 15u) == 0 && ldy % 8 == 0;
  if (dbias || ((dx || dW) && !as_is)) {
    DzArgs a{};
    a.dy = dy;
    a.pre = identity ? nullptr : pre;
    a.ldy = ldy;
    a.T = c.T;
    a.col_blocks = (n + kDzCols - 1) / kDzCols;
    a.ld_dz = up8(n);
    a.n = n;
    if ((dx || dW) && !as_is) {
      a.dz = reinterpret_cast<__nv_bfloat16*>(ws + L.dz);
      oz = {a.dz, a.ld_dz};
    }
    // a single block's sums are db itself
    a.part = !dbias ? nullptr : blocks == 1 ? dbias : reinterpret_cast<float*>(ws + L.db_part);
    const bool vec = n % 8 == 0 && ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(dy) & 15u) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.pre) & 15u) == 0;
    const cudaError_t e = c.out_dtype == MOE_F32 ? launch_dz<float>(a, c.act, vec, stream)
                                                 : launch_dz<__nv_bfloat16>(a, c.act, vec, stream);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  LinearGemm g{};
  g.A = oz.p;
  g.lda = oz.ld;
  g.b_mn = true;
  g.N = c.in_features;
  g.ldc = c.in_features;
  g.act = MOE_ACT_NONE;
  g.status = static_cast<int32_t*>(workspace);
  g.scratch = reinterpret_cast<float*>(ws + L.scratch);
  g.tickets = reinterpret_cast<unsigned*>(ws + kPairTicketOffset);
  if (dbias && blocks > 1) {
    // the first product's shape: its launch adds the partial sums beside it where it can hide them,
    // which saves a launch (about 3 us)
    g.M = dx ? c.T : n;
    g.K = dx ? n : static_cast<int32_t>(c.T);
    g.part = reinterpret_cast<const float*>(ws + L.db_part);
    g.parts = blocks;
    g.part_cols = n;
    if ((dx || dW) && pair_hides_sums(g, device_sm_count()))
      g.db = dbias;
    else if (launch_overlapped(db_kernel, (n + 31) / 32, 1024, 0, stream, 0, g.part, blocks, n, dbias) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (dx) {
    Operand o;
    if (aligned_operand(W, n, c.in_features, row_stride(c.ldw, n, c.in_features), ws + L.w, &o, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    g.B = o.p;
    g.ldb = o.ld;
    g.M = c.T;
    g.K = n;
    g.out_dtype = c.dx_dtype;
    g.C = dx;
    if (launch_linear_pair(g, stream) != cudaSuccess) return MOE_ERR_CUDA;
    g.db = nullptr;
  }
  if (dW) {
    Operand o;
    if (aligned_operand(x, c.T, c.in_features, row_stride(c.ldx, c.T, c.in_features), ws + L.x, &o, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    g.B = o.p;
    g.ldb = o.ld;
    g.a_mn = true;
    g.M = n;
    g.K = static_cast<int32_t>(c.T);
    g.out_dtype = c.dw_dtype;
    g.C = dW;
    if (launch_linear_pair(g, stream) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
