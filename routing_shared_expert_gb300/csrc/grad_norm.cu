// Global norm of a list of gradients and its clipping:
//   norm = (sum over tensors and elements of g^2)^(1/2),  coef = min(1, max_norm / (norm + 1e-6)),
//   out_i = coef g_i.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "share_memory.h"
#include "vec8.cuh"

namespace moe {
namespace {

struct Entry {
  const void* in;
  void* out;
  int64_t rows, cols, ldi, ldo;
  int32_t dtype;
  int16_t lead;           // elements between a 32-byte boundary and the first one
  int16_t vec;            // kReads: gradients in groups of 32 bytes; kWrites: results too
};
constexpr int16_t kReads = 1, kWrites = 2;

// Tensors of one launch: the table is its argument.  60 of them fit into 4 KB; longer lists take a table
// of up to 32 KB.
constexpr int kShortTable = 60, kLongTable = 500;
constexpr int kThreads = 256, kGroups = 4;
constexpr int64_t kChunkBytes = kThreads * kGroups * 32;
__host__ __device__ constexpr int64_t chunk_of(int32_t dtype) { return kChunkBytes / (dtype == MOE_F32 ? 4 : 2); }   // elements
constexpr int kPerSm = 4;
constexpr int kSlots = 152 * kPerSm;  // CTAs, at most: one partial sum each
constexpr size_t kTicketOffset = 64, kPartialOffset = 256;
constexpr size_t kWorkspace = kPartialOffset + kSlots * sizeof(double);

template <int N>
struct Table {
  int32_t chunks, n;
  int32_t first[N];       // number of each tensor's first chunk
  Entry e[N];
};

struct NormSums {
  double* partial;        // [kSlots]
  unsigned* ticket;
  float* norm;
  double max_norm;
  int32_t used;           // slots that earlier launches of this call have written
  int32_t last;           // slots to join after this launch; 0: another launch follows
};

__device__ __forceinline__ float load_elem(const void* p, int32_t dtype, int64_t i) {
  return dtype == MOE_F32 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, int32_t dtype, int64_t i, float v) {
  if (dtype == MOE_F32) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
}

// The tensor that a chunk belongs to: the last one whose first chunk is not after it.
template <int N>
__device__ __forceinline__ int entry_of(const Table<N>& t, int chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (t.first[m] <= chunk) lo = m;
    else hi = m;
  }
  return lo;
}

// A group as it lies in memory: 32 bytes, eight fp32 or 16 bf16.
struct Words {
  uint32_t w[8];
};
__device__ __forceinline__ Words load_words(const void* p) {
  Words r;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
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

// The groups of a chunk: group q of the tensor is its elements G q - lead .. G q - lead + G - 1.  f(words, address
// of the result) takes whole groups, g(i) the elements of groups over the tensor's ends.  Of a dense tensor each
// thread loads all its groups before any is used; a chunk inside the tensor, apart, needs no bounds.
template <typename T, typename F, typename H>
__device__ __forceinline__ void walk_chunk(const Entry& e, int chunk, const F& f, const H& g) {
  constexpr int G = 32 / sizeof(T), kElements = static_cast<int>(kChunkBytes / sizeof(T));
  const int64_t n = e.rows * e.cols, i0 = static_cast<int64_t>(chunk) * kElements - e.lead;
  const T* in = static_cast<const T*>(e.in) + i0;
  const int mine = G * threadIdx.x;
  if (e.rows == 1 && i0 >= 0 && i0 + kElements <= n) {
    Words w[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) w[k] = load_words(in + mine + G * k * kThreads);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) f(w[k], i0 + mine + G * k * kThreads);
  } else if (e.rows == 1) {
    // of the chunk's elements those of the tensor, and of those the whole groups
    const int lo = i0 < 0 ? static_cast<int>(-i0) : 0, hi = static_cast<int>(min(n - i0, int64_t{kElements}));
    const int first = min((lo + G - 1) / G * G, hi), last = max(first, hi / G * G);
    Words w[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int i = mine + G * k * kThreads;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[k].w[j] = 0u;
      if (i >= first && i < last) w[k] = load_words(in + i);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int i = mine + G * k * kThreads;
      if (i >= first && i < last) f(w[k], i0 + i);
    }
    const int j = threadIdx.x;
    if (j < first - lo) g(i0 + lo + j);
    if (j < hi - last) g(i0 + last + j);
  } else {
#pragma unroll 1
    for (int k = 0; k < kGroups; ++k) {      // rows that begin and end on groups
      const int64_t i = i0 + mine + G * k * kThreads;
      if (i + G > n) break;
      const int64_t row = i / e.cols, col = i - row * e.cols;
      f(load_words(static_cast<const T*>(e.in) + row * e.ldi + col), row * e.ldo + col);
    }
  }
}

// One reading of every gradient: 32 bytes per lane and load, four loads on their way, a CTA's sum in fp32 per
// thread (four pairs) and fp64 across threads.  Bound by HBM: 646 M fp32 in 357 us (7.2 TB/s).  Short lists are
// bound by two launches and the join: 16 K values 6.8 us, 1.7 M in ten tensors 11.6 us.
template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm) grad_square_kernel(const __grid_constant__ Table<N> t, NormSums s) {
  __shared__ double part[2][kThreads / 32];
  __shared__ bool join;
  launch_dependents();
  float2 acc[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
  // a CTA's chunks are neighbours: few tensors each
  const int c0 = static_cast<int>(static_cast<int64_t>(t.chunks) * blockIdx.x / gridDim.x),
            c1 = static_cast<int>(static_cast<int64_t>(t.chunks) * (blockIdx.x + 1) / gridDim.x);
  int at = entry_of(t, c0);
  wait_for_previous();
  for (int c = c0; c < c1; ++c) {
    while (at + 1 < t.n && t.first[at + 1] <= c) ++at;
    const Entry& e = t.e[at];
    const int chunk = c - t.first[at];
    auto one = [&](int64_t i) {
      const int64_t row = e.rows == 1 ? 0 : i / e.cols;
      const float v = load_elem(e.in, e.dtype, row * e.ldi + (i - row * e.cols));
      acc[0].x += v * v;
    };
    if (!(e.vec & kReads)) {
      const int64_t i0 = chunk * chunk_of(e.dtype), i1 = min(e.rows * e.cols, i0 + chunk_of(e.dtype));
      for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) one(i);
    } else if (e.dtype == MOE_F32) {
      walk_chunk<float>(e, chunk, [&](const Words& w, int64_t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = make_float2(__uint_as_float(w.w[2 * j]), __uint_as_float(w.w[2 * j + 1]));
          acc[j] = fma2(v, v, acc[j]);
        }
      }, one);
    } else {
      walk_chunk<__nv_bfloat16>(e, chunk, [&](const Words& w, int64_t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j & 3] = fma2(unpack2(w.w[j]), unpack2(w.w[j]), acc[j & 3]);
      }, one);
    }
  }
  const float2 lo = add2(acc[0], acc[1]), hi = add2(acc[2], acc[3]), all = add2(lo, hi);
  const double sum = block_sum_f64(static_cast<double>(all.x) + static_cast<double>(all.y), part[0]);
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

__device__ __forceinline__ void store_scaled(float* p, Words w, float c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) w.w[j] = __float_as_uint(__uint_as_float(w.w[j]) * c);
  store_words(p, w.w);
}
__device__ __forceinline__ void store_scaled(__nv_bfloat16* p, Words w, float c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = mul2(unpack2(w.w[j]), both(c));
    w.w[j] = pack_bf16x2(v.x, v.y);
  }
  store_words(p, w.w);
}

// Each CTA's chunks last to first: what the norm's reading left in L2 is read again before it is replaced.  The gradients
// have to be read twice, since no factor is known before the last one is read: 646 M fp32 take 1167 us with the norm,
// three times their bytes at 6.6 TB/s.
template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm) grad_scale_kernel(const __grid_constant__ Table<N> t, const float* norm) {
  launch_dependents();
  const int c0 = static_cast<int>(static_cast<int64_t>(t.chunks) * blockIdx.x / gridDim.x),
            c1 = static_cast<int>(static_cast<int64_t>(t.chunks) * (blockIdx.x + 1) / gridDim.x);
  int at = entry_of(t, c1 - 1);
  wait_for_previous();
  const float coef = norm[1];
  for (int c = c1 - 1; c >= c0; --c) {
    while (t.first[at] > c) --at;
    const Entry& e = t.e[at];
    const int chunk = c - t.first[at];
    if (coef == 1.f && e.in == e.out) continue;
    auto one = [&](int64_t i) {
      const int64_t row = e.rows == 1 ? 0 : i / e.cols, col = i - row * e.cols;
      store_elem(e.out, e.dtype, row * e.ldo + col, coef * load_elem(e.in, e.dtype, row * e.ldi + col));
    };
    if (!(e.vec & kWrites)) {
      const int64_t i0 = chunk * chunk_of(e.dtype) - e.lead, i1 = min(e.rows * e.cols, i0 + chunk_of(e.dtype));
      for (int64_t i = max(i0, int64_t{0}) + threadIdx.x; i < i1; i += kThreads) one(i);
    } else if (e.dtype == MOE_F32) {
      walk_chunk<float>(e, chunk, [&](const Words& w, int64_t i) { store_scaled(static_cast<float*>(e.out) + i, w, coef); },
                        one);
    } else {
      walk_chunk<__nv_bfloat16>(
          e, chunk, [&](const Words& w, int64_t i) { store_scaled(static_cast<__nv_bfloat16*>(e.out) + i, w, coef); }, one);
    }
  }
}

// ---------------------------------------------------------------------- checks --

constexpr int64_t kMaxElements = int64_t{1} << 40;

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

// What the tensors of a clipping call occupy.
std::vector<Reach> reaches_of(const std::vector<Entry>& list) {
  std::vector<Reach> all;
  all.reserve(2 * list.size());
  for (const Entry& e : list) {
    const uint64_t b = size_of(e.dtype);
    all.push_back(reach_of(e.out, e.rows, e.cols * b, e.ldo * b, true));
    if (e.in != e.out || e.ldi != e.ldo) all.push_back(reach_of(e.in, e.rows, e.cols * b, e.ldi * b, false));
  }
  return all;
}

template <int N>
cudaError_t launch_lists(const std::vector<Entry>& list, NormSums sums, bool clip, cudaStream_t s) {
  const size_t n = list.size();
  Table<N> t;
  auto fill = [&](size_t at, bool reads) {
    t.n = static_cast<int32_t>(std::min<size_t>(N, n - at));
    int64_t chunks = 0;
    for (int32_t i = 0; i < t.n; ++i) {
      t.e[i] = list[at + i];
      if (reads && t.e[i].ldi == t.e[i].cols) {      // a dense gradient, whatever its result is: the same sums
        t.e[i].cols *= t.e[i].rows;
        t.e[i].rows = 1;
      }
      t.first[i] = static_cast<int32_t>(chunks);
      const int64_t size = chunk_of(t.e[i].dtype);
      chunks += (t.e[i].lead + t.e[i].rows * t.e[i].cols + size - 1) / size;
    }
    t.chunks = static_cast<int32_t>(chunks);     // 2^40 elements at most: 2^27 chunks, and one more per tensor
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>({chunks, kSlots, int64_t{kPerSm} * device_sm_count()})));
  };
  size_t at = 0;
  do {   // a list without elements has one launch too, for the norm of nothing
    const unsigned grid = fill(at, true);
    at += t.n;
    const int32_t slots = std::max(sums.used, static_cast<int32_t>(grid));
    if (at >= n) sums.last = slots;
    const cudaError_t e = launch_over(grad_square_kernel<N>, dim3(grid), kThreads, 0, s, t, sums);
    if (e != cudaSuccess) return e;
    sums.used = slots;
  } while (at < n);
  if (!clip) return cudaSuccess;
  // the tables last to first, as the chunks
  for (size_t tables = (n + N - 1) / N; tables > 0; --tables) {
    const unsigned grid = fill((tables - 1) * N, false);
    const cudaError_t e = launch_over(grad_scale_kernel<N>, dim3(grid), kThreads, 0, s, t, static_cast<const float*>(sums.norm));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
    // in groups: dense from any element on, or rows that begin and end on groups
    const int64_t b = static_cast<int64_t>(size_of(e.dtype)), G = 32 / b;
    const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(e.in) % 32) / b,
                  lead_out = static_cast<int64_t>(reinterpret_cast<uintptr_t>(e.out) % 32) / b;
    const bool rows = lead == 0 && e.cols % G == 0 && e.ldi % G == 0;
    if (e.ldi == e.cols) e.lead = static_cast<int16_t>(lead);
    if (e.ldi == e.cols || rows) e.vec = kReads;
    if (lead_out == lead && (e.rows == 1 || (rows && e.ldo % G == 0))) e.vec |= kWrites;
    list.push_back(e);
  }
  if (reinterpret_cast<uintptr_t>(norm) & 3u || reinterpret_cast<uintptr_t>(workspace) & 255u)
    return MOE_ERR_MISALIGNED;
  std::vector<Reach> reaches;
  if (clip) reaches = reaches_of(list);
  if (any_written_is_shared(reaches)) return MOE_ERR_INVALID_ARG;
  if (bytes < kWorkspace) return MOE_ERR_WORKSPACE_TOO_SMALL;
  // the norm is written before the gradients are read again
  for (const Reach& r : reaches)
    if (share_memory(r, reach_of(norm, 1, 8, 8, true))) return MOE_ERR_INVALID_ARG;

  NormSums sums{};
  sums.partial = reinterpret_cast<double*>(static_cast<char*>(workspace) + kPartialOffset);
  sums.ticket = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kTicketOffset);
  sums.norm = norm;
  sums.max_norm = max_norm;
  const cudaError_t e = list.size() <= kShortTable ? launch_lists<kShortTable>(list, sums, clip, s)
                                                   : launch_lists<kLongTable>(list, sums, clip, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
