// Groups of eight consecutive values: asynchronous copies to shared memory (16-byte pieces: one for
// bf16, two for fp32), and one 16- or 32-byte store.
#pragma once

#include "common.cuh"

namespace moe {

template <typename T>
constexpr int kPieces = static_cast<int>(sizeof(T)) / 2;   // 16-byte pieces of a group

__device__ __forceinline__ void unpack_bf16x8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The bytes of a tensor with rows ld elements apart: what may be read.
struct Extent {
  uintptr_t lo, hi;
};
__device__ __forceinline__ Extent extent_of(const void* p, int64_t rows, int64_t ld, int64_t cols, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(((rows - 1) * ld + cols) * elem)};
}

// Begins the copy of elements [e0, e0 + 8) of a row of d to a thread's own pieces in shared memory,
// `stride` bytes apart.  The group is aligned to its size; one that reaches over an end of the row is
// copied whole, the neighbouring rows' values with it, and element by element only at the
// tensor's own ends.  Values outside the row are for the reader to leave out.
template <typename T>
__device__ __forceinline__ void copy_group(char* dst, uint32_t stride, const T* row, int e0, int d, const Extent& t) {
  if (e0 + 8 <= 0 || e0 >= d) return;
  const char* src = reinterpret_cast<const char*>(row + e0);
  const uintptr_t a = reinterpret_cast<uintptr_t>(src);
  if (a >= t.lo && a + 8 * sizeof(T) <= t.hi) {
#pragma unroll
    for (int i = 0; i < kPieces<T>; ++i) cp_async16(smem_u32(dst) + i * stride, src + 16 * i, 16);
    return;
  }
#pragma unroll 1
  for (int j = max(0, -e0); j < min(8, d - e0); ++j) {
    constexpr int per = 16 / static_cast<int>(sizeof(T));
    *reinterpret_cast<T*>(dst + j / per * stride + j % per * sizeof(T)) = row[e0 + j];
  }
}
__device__ __forceinline__ void read_group(const char* src, uint32_t, const __nv_bfloat16*, float (&v)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(src), v);
}
__device__ __forceinline__ void read_group(const char* src, uint32_t stride, const float*, float (&v)[8]) {
  const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + stride);
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}
__device__ __forceinline__ bool whole_group(int e0, int d) { return e0 >= 0 && e0 + 8 <= d; }
__device__ __forceinline__ void clear_outside(float (&v)[8], int e0, int d) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (e0 + j < 0 || e0 + j >= d) v[j] = 0.f;
}
template <typename T>
__device__ __forceinline__ void store_group(T* row, int e0, int d, const float (&v)[8]) {
  if (whole_group(e0, d)) {
    store8(row + e0, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j >= 0 && e0 + j < d) row[e0 + j] = from_f32<T>(v[j]);
  }
}

}  // namespace moe
