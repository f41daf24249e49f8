// Global norm of a list of gradients and its clipping:
//   norm = (sum over tensors and elements of g^2)^(1/2),  coef = min(1, max_norm / (norm + 1e-6)),
//   out_i = coef g_i.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

struct Entry {
  const void* in;
  void* out;
  int64_t rows, cols, ldi, ldo;
  int64_t first;          // number of the tensor's first chunk
  int32_t dtype;
};

constexpr int kEntries = 56;          // tensors of one launch: the table is its argument (< 4 KB)
constexpr int kThreads = 256;
constexpr int64_t kChunk = 8192;      // elements
constexpr int kSlots = 152 * 8;       // CTAs, at most: one partial sum each
constexpr size_t kTicketOffset = 64, kPartialOffset = 256;
constexpr size_t kWorkspace = kPartialOffset + kSlots * sizeof(double);

struct Table {
  Entry e[kEntries];
  int32_t n;
  int64_t chunks;
};

struct NormSums {
  double* partial;        // [kSlots]
  unsigned* ticket;
  float* norm;
  double max_norm;
  int32_t used;           // slots that earlier launches of this call have written
  int32_t last;           // slots to join after this launch; 0: another launch follows
};

__device__ __forceinline__ const Entry& entry_of(const Table& t, int64_t chunk) {
  int lo = 0, hi = t.n;   // the last tensor whose first chunk is not after this one
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (t.e[m].first <= chunk) lo = m;
    else hi = m;
  }
  return t.e[lo];
}

__device__ __forceinline__ float load_elem(const void* p, int32_t dtype, int64_t i) {
  return dtype == MOE_F32 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ double block_sum_f64(double v, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

__global__ void __launch_bounds__(kThreads) grad_square_kernel(const __grid_constant__ Table t, NormSums s) {
  __shared__ double part[2][kThreads / 32];
  __shared__ bool join;
  float acc = 0.f;
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    const Entry& e = entry_of(t, chunk);
    const int64_t n = e.rows * e.cols, i0 = (chunk - e.first) * kChunk, i1 = min(n, i0 + kChunk);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const int64_t row = e.rows == 1 ? 0 : i / e.cols;
      const float v = load_elem(e.in, e.dtype, row * e.ldi + (i - row * e.cols));
      acc += v * v;
    }
  }
  const double sum = block_sum_f64(acc, part[0]);
  if (threadIdx.x == 0) {
    s.partial[blockIdx.x] = sum + (blockIdx.x < s.used ? s.partial[blockIdx.x] : 0.0);
    __threadfence();
    join = s.last && atomicAdd(s.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!join) return;
  // the last CTA joins the slots in order
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < s.last; i += kThreads) v += __ldcg(s.partial + i);
  v = block_sum_f64(v, part[1]);
  if (threadIdx.x == 0) {
    const double norm = sqrt(v);
    double coef = isinf(s.max_norm) ? 1.0 : s.max_norm / (norm + 1e-6);
    if (coef > 1.0) coef = 1.0;      // a NaN stays
    s.norm[0] = static_cast<float>(norm);
    s.norm[1] = static_cast<float>(coef);
    *s.ticket = 0;
  }
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Table t, const float* norm) {
  const float coef = norm[1];
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    const Entry& e = entry_of(t, chunk);
    if (coef == 1.f && e.in == e.out) continue;
    const int64_t n = e.rows * e.cols, i0 = (chunk - e.first) * kChunk, i1 = min(n, i0 + kChunk);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const int64_t row = e.rows == 1 ? 0 : i / e.cols, col = i - row * e.cols;
      const float v = coef * load_elem(e.in, e.dtype, row * e.ldi + col);
      if (e.dtype == MOE_F32) static_cast<float*>(e.out)[row * e.ldo + col] = v;
      else static_cast<__nv_bfloat16*>(e.out)[row * e.ldo + col] = from_f32<__nv_bfloat16>(v);
    }
  }
}

// ---------------------------------------------------------------------- checks --

constexpr int64_t kMaxElements = int64_t{1} << 40;

struct Extent {
  uintptr_t lo, hi;       // bytes spanned
  uint64_t pitch, width;  // bytes between rows (0: one row) and of a row
  int32_t tensor;
  bool written;
};

bool share_memory(const Extent& a, const Extent& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  // columns of rows of one matrix: apart when they are apart within a row
  const uint64_t gap = (b.lo >= a.lo ? b.lo - a.lo : a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
  return !(gap >= a.width && gap + b.width <= a.pitch);
}

bool elem_ok(const moe_tensor& t) {
  return (t.dtype == MOE_F32 || t.dtype == MOE_BF16) && t.rows >= 0 && t.cols >= 0;
}
uint64_t size_of(int32_t t) { return t == MOE_F32 ? 4 : 2; }

moe_status check_tensor(const moe_tensor& t, Entry& e, bool out) {
  if (!elem_ok(t)) return MOE_ERR_INVALID_ARG;
  const int64_t ld = t.rows > 1 && t.ld ? t.ld : t.cols;
  if (ld < t.cols) return MOE_ERR_INVALID_ARG;
  if (t.rows > 0 && t.cols > 0) {
    if (t.rows > kMaxElements || ld > kMaxElements / t.rows) return MOE_ERR_UNSUPPORTED;
    if (!t.data) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t.data) & (size_of(t.dtype) - 1)) return MOE_ERR_MISALIGNED;
  }
  if (out) {
    e.out = t.data;
    e.ldo = ld;
  } else {
    e.in = t.data;
    e.ldi = ld;
    e.rows = t.rows;
    e.cols = t.cols;
    e.dtype = t.dtype;
  }
  return MOE_OK;
}

Extent extent_of(const void* p, const Entry& e, int64_t ld, int32_t i, bool written) {
  const uint64_t b = size_of(e.dtype);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + ((e.rows - 1) * ld + e.cols) * b, e.rows > 1 ? ld * b : 0, e.cols * b, i, written};
}

// Whether tensors that are written share memory with each other or with one that is read.
bool overlap(const std::vector<Entry>& list) {
  std::vector<Extent> x, open;
  for (size_t i = 0; i < list.size(); ++i) {
    const Entry& e = list[i];
    const bool same = e.in == e.out && e.ldi == e.ldo;
    x.push_back(extent_of(e.out, e, e.ldo, static_cast<int32_t>(i), true));
    if (!same) x.push_back(extent_of(e.in, e, e.ldi, static_cast<int32_t>(i), false));
  }
  std::sort(x.begin(), x.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  for (const Extent& e : x) {
    size_t k = 0;
    for (const Extent& o : open) {
      if (o.hi <= e.lo) continue;
      if ((o.written || e.written) && share_memory(o, e)) return true;
      open[k++] = o;
    }
    open.resize(k);
    open.push_back(e);
  }
  return false;
}

moe_status run_norm(const moe_tensor* grads, const moe_tensor* out, int32_t count, double max_norm, float* norm,
                    bool clip, void* workspace, size_t bytes, cudaStream_t s) {
  if (count < 0 || count > (1 << 20) || (count > 0 && !grads) || !norm || !workspace || !(max_norm >= 0.0))
    return MOE_ERR_INVALID_ARG;
  std::vector<Entry> list;
  list.reserve(static_cast<size_t>(count));
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    Entry e{};
    moe_status st = check_tensor(grads[i], e, false);
    if (st != MOE_OK) return st;
    if (clip) {
      const moe_tensor& o = out ? out[i] : grads[i];
      if (o.rows != e.rows || o.cols != e.cols || o.dtype != e.dtype) return MOE_ERR_INVALID_ARG;
      st = check_tensor(o, e, true);
      if (st != MOE_OK) return st;
    }
    if (e.rows == 0 || e.cols == 0) continue;
    total += e.rows * e.cols;
    if (total > kMaxElements) return MOE_ERR_UNSUPPORTED;
    if (e.ldi == e.cols && (!clip || e.ldo == e.cols)) {   // dense: one row
      e.cols *= e.rows;
      e.rows = 1;
      e.ldi = e.ldo = e.cols;
    }
    list.push_back(e);
  }
  if (reinterpret_cast<uintptr_t>(norm) & 3u || reinterpret_cast<uintptr_t>(workspace) & 255u)
    return MOE_ERR_MISALIGNED;
  if (bytes < kWorkspace) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (clip && overlap(list)) return MOE_ERR_INVALID_ARG;

  NormSums sums{};
  sums.partial = reinterpret_cast<double*>(static_cast<char*>(workspace) + kPartialOffset);
  sums.ticket = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kTicketOffset);
  sums.norm = norm;
  sums.max_norm = max_norm;
  const size_t n = list.size();
  auto fill = [&](size_t at, Table& t) {
    t.n = static_cast<int32_t>(std::min<size_t>(kEntries, n - at));
    t.chunks = 0;
    for (int32_t i = 0; i < t.n; ++i) {
      t.e[i] = list[at + i];
      t.e[i].first = t.chunks;
      t.chunks += (t.e[i].rows * t.e[i].cols + kChunk - 1) / kChunk;
    }
    return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(t.chunks, kSlots)));
  };
  size_t at = 0;
  do {   // a list without elements has one launch too, for the norm of nothing
    Table t{};
    const int32_t grid = fill(at, t);
    at += t.n;
    if (at >= n) sums.last = std::max(sums.used, grid);
    grad_square_kernel<<<grid, kThreads, 0, s>>>(t, sums);
    sums.used = std::max(sums.used, grid);
  } while (at < n);
  if (clip)
    for (at = 0; at < n; at += kEntries) {
      Table t{};
      const int32_t grid = fill(at, t);
      grad_scale_kernel<<<grid, kThreads, 0, s>>>(t, norm);
    }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status guarded(const moe_tensor* grads, const moe_tensor* out, int32_t count, double max_norm, float* norm,
                   bool clip, void* workspace, size_t bytes, cudaStream_t s) {
  try {
    return run_norm(grads, out, count, max_norm, norm, clip, workspace, bytes, s);
  } catch (...) {        // host memory for the list
    return MOE_ERR_UNSUPPORTED;
  }
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_grad_norm_workspace_size(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = moe::kWorkspace;
  return MOE_OK;
}

moe_status moe_grad_norm(const moe_tensor* grads, int32_t count, float max_norm, float* norm,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return moe::guarded(grads, nullptr, count, max_norm, norm, false, workspace, workspace_bytes, stream);
}

moe_status moe_clip_grad_norm(const moe_tensor* grads, const moe_tensor* out, int32_t count,
                              float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  return moe::guarded(grads, out, count, max_norm, norm, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
