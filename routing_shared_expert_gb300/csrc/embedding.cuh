// Token embedding: what the lookup and the gradient of the table share.
#pragma once

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "load_any.cuh"
#include "vec8.cuh"

namespace moe {

struct EmbedArgs {
  const void* ids;
  const void* src;       // table, or dout
  void* dst;             // out, or dtable
  int64_t T, V, ldt, ldo;
  int32_t d, accumulate;
  float scale;
  int32_t* status;
  char* scratch;         // of the gradient: the workspace past its header
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

// Eight values of a row from any element's address on, elements [e0, e0 + 8) of which [0, d) are wanted.
template <typename T>
__device__ __forceinline__ void take_any(const T* p, int e0, int d, const Span& span, float2 (&v)[4]) {
  const int skip = max(0, -e0), valid = min(8, d - e0);
  float u[8];
  if (skip == 0) {
    take8(load8_raw(p, span), p, valid, u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = j >= skip && j < valid ? to_f32(p[j]) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(u[2 * j], u[2 * j + 1]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) { store_whole(p, v); }
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0].x), "f"(v[0].y),
               "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
               : "memory");
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p) : "memory");
}
__device__ __forceinline__ void load8(const float* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint32_t (&w)[8], float2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = sizeof(T) == 4 ? make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1])) : unpack2(w[j]);
}

constexpr int kColumns = 256;      // of a warp at a time

// A lane's eight columns of a warp's slice, which begins at column c0: neighbours where rows begin on groups of
// eight (ALIGNED), else 32 apart, so that neighbouring lanes read and write neighbouring values.
template <bool ALIGNED>
__device__ __forceinline__ int column(int c0, int j) {
  const int lane = threadIdx.x & 31;
  return ALIGNED ? c0 + 8 * lane + j : c0 + 32 * j + lane;
}
__device__ __forceinline__ float& value(float2 (&v)[4], int j) { return j & 1 ? v[j / 2].y : v[j / 2].x; }

template <typename T, bool ALIGNED>
struct Slice {      // as it is loaded
  uint32_t w[8];
  __device__ __forceinline__ void load(const T* row, int c0, int d) {
    if (ALIGNED) {
      if (column<true>(c0, 0) < d) load8(row + column<true>(c0, 0), w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = column<false>(c0, j);
        if (sizeof(T) == 4) w[j] = c < d ? *reinterpret_cast<const uint32_t*>(row + c) : 0u;
        else w[j] = c < d ? *reinterpret_cast<const uint16_t*>(row + c) : 0u;
      }
    }
  }
  __device__ __forceinline__ void unpack(float2 (&v)[4]) const {
    if (ALIGNED) {
      unpack8<T>(w, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) value(v, j) = __uint_as_float(sizeof(T) == 4 ? w[j] : w[j] << 16);
    }
  }
};
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_slice(T* row, int c0, int d, float2 (&v)[4]) {
  if (ALIGNED) {
    if (column<true>(c0, 0) < d) store8(row + column<true>(c0, 0), v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (column<false>(c0, j) < d) row[column<false>(c0, j)] = from_f32<T>(value(v, j));
  }
}

// Whether rows begin and end on groups of eight values (host).
template <typename T>
bool groups_of_eight(const void* p, int64_t ld, int32_t d) {
  return reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0 && ld % 8 == 0 && d % 8 == 0;
}

// The gradient of the table (embedding_grad.cu), and the scratch memory that it takes.
size_t embedding_scratch(int64_t T, int64_t V, int32_t d);
cudaError_t launch_embedding_backward(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s);

}  // namespace moe
