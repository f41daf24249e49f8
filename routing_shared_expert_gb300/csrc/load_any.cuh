// Eight neighbouring values of a row from any element's address, in 16-byte loads.
//
// A row of an odd stride starts anywhere; its values are then taken from the two (bf16) or three
// (fp32) aligned 16-byte pieces that hold them and moved into place, the neighbouring lanes' pieces
// coming from L1.  Value by value the same reads are eight load instructions, each touching every
// cache line of the warp's 512 or 1024 bytes.  The gradients of 3000 x 2048 to 2049 in fp32: 122 -> 69
// us; of 16995 x 87 to 6133 in bf16, together with narrower tiles: 282 -> 234 us; one token of
// 4095 x 8192: 37 -> 29 us.  The copies to aligned rows, which do nothing else, gain nothing from
// it (1023 x 4093 to 4096: 41 -> 44 us) and read value by value.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace moe {

// The bytes that a tensor spans, gaps between its rows included: what may be read.
struct Span {
  uintptr_t lo, hi;
};
__device__ __forceinline__ Span span_of(const void* p, int64_t rows, int64_t ld, int64_t cols, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(((rows - 1) * ld + cols) * elem)};
}

// The aligned pieces that hold the eight values from p on.  Loading is apart from using them, and has
// no branch, so that several pieces can be on their way.
struct Raw8 {
  uint4 piece[3];            // the third only for fp32
  bool whole;                // all of those that are needed lie in the span
};
template <typename T>
__device__ __forceinline__ Raw8 load8_raw(const T* p, const Span& s) {
  constexpr int N = sizeof(T) == 2 ? 1 : 2;   // pieces of eight values
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), base = a & ~uintptr_t{15};
  const uint4* q = reinterpret_cast<const uint4*>(base);
  const bool off = a != base;
  Raw8 r;
  r.whole = base >= s.lo && base + 16 * (off ? N + 1 : N) <= s.hi;
#pragma unroll
  for (int i = 0; i < N + 1; ++i) {
    r.piece[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r.whole && (i < N || off)) r.piece[i] = q[i];
  }
  return r;
}

// Values 0 .. 7 from p on as four words of two; zeros from `valid` on.
__device__ __forceinline__ uint4 take8(const Raw8& r, const __nv_bfloat16* p, int valid) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
  const uint4 u = r.piece[0], v = r.piece[1];
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t x[6], y[5], o[4];
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) y[i] = off & 4 ? x[i + 1] : x[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(y[i], y[i + 1], (off & 2) * 8);
  if (!r.whole) {   // at the tensor's ends
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < valid ? h[2 * i] : 0u;
      const uint32_t hi = 2 * i + 1 < valid ? h[2 * i + 1] : 0u;
      o[i] = lo | hi << 16;
    }
  } else if (valid < 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = valid > 2 * i + 1 ? o[i] : valid > 2 * i ? o[i] & 0xffffu : 0u;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void take8(const Raw8& r, const __nv_bfloat16* p, int valid, float (&v)[8]) {
  const uint4 u = take8(r, p, valid);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void take8(const Raw8& r, const float* p, int valid, float (&v)[8]) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
  const uint4 t = r.piece[0], u = r.piece[1], z = r.piece[2];
  const uint32_t w[12] = {t.x, t.y, t.z, t.w, u.x, u.y, u.z, u.w, z.x, z.y, z.z, z.w};
  uint32_t x[9];
#pragma unroll
  for (int i = 0; i < 9; ++i) x[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(off & 4 ? x[i + 1] : x[i]);
  if (!r.whole) {   // at the tensor's ends
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? p[i] : 0.f;
  } else if (valid < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? v[i] : 0.f;
  }
}

}  // namespace moe
