// Groups of G = 4 or 8 consecutive values as pairs: asynchronous copies to shared memory, one of 8 or 16
// bytes each, arithmetic on pairs (one instruction for two values), and one store each.
//
// G is 8 where every operand is bf16 and 4 where one is fp32: a lane's copy is then at most 16 bytes and a
// warp's copies are one run of memory.  (Eight fp32 in two copies of 16 bytes ask L2 for every 32-byte
// sector twice.)
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void store_whole(__nv_bfloat16* p, const float2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                            pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ void store_whole(__nv_bfloat16* p, const float2 (&v)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
}
__device__ __forceinline__ void store_whole(float* p, const float2 (&v)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}

// The pairs rounded to T and back.
template <typename T, int N>
__device__ __forceinline__ void round_to(float2 (&v)[N]) {
  if (sizeof(T) == 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = unpack2(pack_bf16x2(v[i].x, v[i].y));
}

// Begins the copy of a group that lies in its row.
template <int G, typename T>
__device__ __forceinline__ void copy_whole(char* dst, const T* src) {
  static_assert(G * sizeof(T) == 16 || G * sizeof(T) == 8, "a group is one copy");
  if (G * sizeof(T) == 16) cp_async16(smem_u32(dst), src, 16);
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// The same of the elements of a group that `mask` has, for the groups at a tensor's own ends, whose other
// elements may not be read.
template <int G, typename T>
__device__ __noinline__ void copy_masked(char* dst, const T* src, unsigned mask) {
  T v[G];
#pragma unroll
  for (int j = 0; j < G; ++j) v[j] = mask >> j & 1 ? src[j] : from_f32<T>(0.f);
#pragma unroll
  for (int j = 0; j < G; ++j) reinterpret_cast<T*>(dst)[j] = v[j];
}
template <int G, typename T>
__device__ __forceinline__ void clear_group(char* at) {
  if (G * sizeof(T) == 16) *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
  else *reinterpret_cast<uint2*>(at) = make_uint2(0u, 0u);
}
// Zeros where the mask has none.
template <int N>
__device__ __forceinline__ void keep(float2 (&v)[N], unsigned mask) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = make_float2(mask >> 2 * j & 1 ? v[j].x : 0.f, mask >> 2 * j & 2 ? v[j].y : 0.f);
}
__device__ __forceinline__ void read_group(const char* src, const __nv_bfloat16*, float2 (&v)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(src);
  v[0] = unpack2(u.x), v[1] = unpack2(u.y), v[2] = unpack2(u.z), v[3] = unpack2(u.w);
}
__device__ __forceinline__ void read_group(const char* src, const __nv_bfloat16*, float2 (&v)[2]) {
  const uint2 u = *reinterpret_cast<const uint2*>(src);
  v[0] = unpack2(u.x), v[1] = unpack2(u.y);
}
__device__ __forceinline__ void read_group(const char* src, const float*, float2 (&v)[2]) {
  const float4 u = *reinterpret_cast<const float4*>(src);
  v[0] = make_float2(u.x, u.y), v[1] = make_float2(u.z, u.w);
}
// Stores the elements that the mask has.  In line: a call here is on the way of every row (16384 x 4095 76 us, called
// 84), while one at a tensor's own ends above is not (in line 98: its instructions would be predicated ones in
// every thread).
template <typename T, int N>
__device__ __forceinline__ void store_masked(T* dst, unsigned mask, const float2 (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (mask >> 2 * j & 1) dst[2 * j] = from_f32<T>(v[j].x);
    if (mask >> 2 * j & 2) dst[2 * j + 1] = from_f32<T>(v[j].y);
  }
}

}  // namespace moe
