// Normalisation of rows, LAYER or RMS: what the forward and the backward pass share.
//
//   h = x + r,  mean = sum h / d,  rstd = (sum (h - mean)^2 / d + eps)^(-1/2),  y = (h - mean) rstd w + b
//   xhat = (h - mean) rstd,  g = dy w,
//   dx = rstd (g - sum g / d - xhat sum (g xhat) / d) + dsum,  dw = sum_t dy xhat,  db = sum_t dy
// (RMS: mean = 0, no sum g).  The variance is taken from deviations, never as E h^2 - mean^2.
#pragma once

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "row_ends.h"
#include "row_reduce.cuh"
#include "vec8.cuh"

namespace moe {

struct NormArgs {
  const void* x;        // h in the backward pass
  const void* r;        // residual, or dsum
  const void* w;
  const void* b;
  void* s;              // sum, or dx
  void* y;              // dy in the backward pass (read only)
  float* mean;
  float* rstd;
  float* partial;       // [slots][2][d]
  float* dw;
  float* db;
  int64_t T, ldx, ldr, lds, ldy;
  int32_t d, slots;
  float eps;
  int32_t rms, w_dtype;
  int32_t lanes;        // threads of a team, which takes a row at a time
  int32_t stages;       // turns whose rows are on their way, 1 to 4
  int32_t room;         // rows at either end of the operands whose groups over a row's end are not copied whole
};

__device__ __forceinline__ float load_param(const void* p, int32_t dtype, int32_t c, float none) {
  if (!p) return none;
  return dtype == MOE_F32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const __nv_bfloat16*>(p)[c]);
}

// The gradients of rows h of X with dy of Y, dsum and dx of the given type (layernorm_grad.cuh).
template <typename X, typename Y>
cudaError_t launch_layernorm_grad(const NormArgs& a, int32_t stream_dtype, cudaStream_t s);

// --------------------------------------------------------------- rows in groups --
// Rows whose operands all start at the same place within a group of G elements (aligned tensors
// with one width or stride, odd ones included): a thread takes P groups, E = P G elements.  A row
// that starts `phase` elements into a group has two end groups that are not whole.  A CTA is several
// teams of `lanes` threads, each with rows of its own, and one copy of the parameters in shared memory.
// Its rows are gridDim.x apart, a multiple of eight unless the stride is one, so that the phase is the
// same for all of them and the parameters can lie at that phase.  SPLIT: a team is a power of two of a
// warp's lanes; else it is whole warps with a barrier of their own.  ENDS: rows may begin or end within a
// group; else every group lies in its row or past it.
//
// Each thread copies its own groups of the next rows asynchronously into its own slots of a ring in
// shared memory, a.stages rows ahead: the bytes on their way do not depend on registers, and the
// ring needs no barrier.

constexpr int kMaxTeams = 8;     // of whole warps: barriers 1 to 8
constexpr size_t kStaticSmem = 4 * 1024;      // the kernels' own arrays, at most

template <typename X, typename S, typename Y>
constexpr int kGroup = sizeof(X) + sizeof(S) + sizeof(Y) == 6 ? 8 : 4;

// Pairs `from` .. from + M - 1 of group q of a parameter in shared memory.  G = 8: the lower and the upper half of all
// groups lie apart, so that neighbouring lanes' 16-byte reads are neighbours.
template <int M>
__device__ __forceinline__ void param_values(const float* p, int groups, int q, int from, float2 (&v)[M]) {
#pragma unroll
  for (int i = 0; i < M; i += 2) {
    const float4 u = reinterpret_cast<const float4*>(p)[(from + i) / 2 * groups + q];
    v[i] = make_float2(u.x, u.y), v[i + 1] = make_float2(u.z, u.w);
  }
}
template <int N>
__device__ __forceinline__ void param_group(const float* p, int groups, int q, float2 (&v)[N]) {
  param_values(p, groups, q, 0, v);
}
template <int G>
__device__ __forceinline__ void stage_param(float* dst, const void* src, int32_t dtype, int groups, int phase, int d) {
  const bool pieces = (reinterpret_cast<uintptr_t>(src) & 15) == 0 && phase == 0;    // 16 bytes at a time
#pragma unroll 4
  for (int q = threadIdx.x; q < groups; q += blockDim.x) {
    float v[G];
    const int c0 = G * q - phase;
    if (pieces && c0 + G <= d && dtype == MOE_F32) {
#pragma unroll
      for (int j = 0; j < G; j += 4) {
        const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + c0 + j);
        v[j] = u.x, v[j + 1] = u.y, v[j + 2] = u.z, v[j + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] = c0 + j >= 0 && c0 + j < d ? load_param(src, dtype, c0 + j, 0.f) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < G; j += 4)
      reinterpret_cast<float4*>(dst)[j / 4 * groups + q] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}
template <int G, typename T>
__device__ __forceinline__ int phase_of(const T* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (G - 1);
}
__device__ __forceinline__ void wait_stage(int stages) {   // the oldest of `stages` copies has landed
  if (stages == 1) cp_async_wait<0>();
  else if (stages == 2) cp_async_wait<1>();
  else if (stages == 3) cp_async_wait<2>();
  else cp_async_wait<3>();
}

// Where a thread stands.  R: rows that a team takes at a time.
template <int G, int P, bool SPLIT, int R = 1>
struct Seat {
  int lanes, lane, team, groups, phase;
  int row, step;      // the team's first row, and from one to the next
  int turns;          // of its warp, the last of which may be past the last row for some teams (SPLIT) and rows (R)
  int e0;             // first element of the first group within the row, the others G * lanes further
  unsigned mask[P];   // which elements of each group lie in the row
  bool whole[P];      // all of them,
  bool part[P];       // some but not all (ENDS only)
  bool all;           // whether all groups are whole
  __device__ __forceinline__ Seat(const NormArgs& a, int first_phase) {
    lanes = a.lanes;
    team = threadIdx.x / lanes;
    lane = threadIdx.x - team * lanes;
    groups = lanes * P;
    phase = first_phase;
    row = blockIdx.x + team * gridDim.x;
    step = blockDim.x / lanes * gridDim.x;
    const int first = SPLIT ? blockIdx.x + (threadIdx.x & ~31) / lanes * gridDim.x : row, T = static_cast<int>(a.T);
    turns = first < T ? (T - first + R * step - 1) / (R * step) : 0;
    e0 = G * lane - phase;
    all = true;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      mask[k] = 0;
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (column(k) + j >= 0 && column(k) + j < a.d) mask[k] |= 1u << j;
      whole[k] = column(k) >= 0 && column(k) + G <= a.d;
      part[k] = !whole[k] && mask[k] != 0;
      all = all && whole[k];
    }
  }
  __device__ __forceinline__ int column(int k) const { return e0 + k * G * lanes; }
};

// A thread's groups of one operand: `at` is where the current row's lie in the ring, copies of later rows
// begin from `next`.  The pieces are `stride` bytes apart.
template <typename T_, int G, int P, bool ENDS>
struct Feed {
  const T_* next;      // element 0 of the thread's first group, in the row to be copied next
  int64_t step;       // elements to the team's row after it
  uint32_t stride;
  template <typename At>
  __device__ __forceinline__ Feed(const void* base, int64_t ld, const At& s)
      : next(static_cast<const T_*>(base) + s.row * ld + s.e0), step(s.step * ld),
        stride(blockDim.x * static_cast<uint32_t>(G * sizeof(T_))) {}
  // The row's groups begin their way.  One over an end of the row is copied whole, what lies beside the row with it,
  // but for the groups that could leave the tensor (row_ends.h).
  template <typename At>
  __device__ __forceinline__ void copy(char* to, const At& s, int at, int T, int room) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const T_* src = next + k * G * s.lanes;
      const bool inside = ENDS && s.part[k] && copied_whole(at, T, room, s.mask[k], G);
      if (s.whole[k] || inside) copy_whole<G>(to + k * stride, src);
      else if (ENDS && s.part[k]) copy_masked<G>(to + k * stride, src, s.mask[k]);
    }
    next += step;
  }
  // Zeros in the places of groups past the row, which are never copied.  (Where rows end on groups the masks stay out of
  // it: with them the gradients of 32768 x 4096 took 134 us, not 129.)
  template <typename At>
  __device__ __forceinline__ void clear_unused(char* at, const At& s) {
#pragma unroll
    for (int k = 0; k < P; ++k)
      if (ENDS ? s.mask[k] == 0 : !s.whole[k]) clear_group<G, T_>(at + k * stride);
  }
  __device__ __forceinline__ void clear(char* at) {
#pragma unroll
    for (int k = 0; k < P; ++k) clear_group<G, T_>(at + k * stride);
  }
  // Group k, with zeros outside the row.
  template <typename At>
  __device__ __forceinline__ void read(const char* at, int k, const At& s, float2 (&v)[G / 2]) const {
    read_group(at + k * stride, static_cast<const T_*>(nullptr), v);
    if (ENDS && s.part[k]) {
      asm volatile("");      // a branch that few threads take, not selections in all of them
      keep(v, s.mask[k]);
    }
  }
};

// A thread's groups of a result, row by row.
template <typename T, int G, int P, bool ENDS>
struct Sink {
  T* row;
  int64_t step;
  template <typename At>
  __device__ __forceinline__ Sink(void* base, int64_t ld, const At& s)
      : row(static_cast<T*>(base) + s.row * ld + s.e0), step(s.step * ld) {}
  // Group k of the row that is `ahead` elements further.
  template <typename At>
  __device__ __forceinline__ void store(int k, const At& s, const float2 (&v)[G / 2], int64_t ahead = 0) {
    T* dst = row + ahead + k * G * s.lanes;
    if (s.whole[k]) store_whole(dst, v);
    else if (ENDS && s.part[k]) store_masked(dst, s.mask[k], v);
  }
};

template <bool SPLIT, int N, int W>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part, int& turn, int lanes, int lane, int team) {
  if (SPLIT) {
    for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else {
    team_sum<N, W>(v, part + (2 * team + turn) * N * W, lane >> 5, lanes >> 5, 1 + team);
    turn ^= 1;
  }
}

// ------------------------------------------------------------------ launch plan --

constexpr size_t kSharedPerSm = 227 * 1024, kDefaultSmem = 48 * 1024;

// Rows of room for the operands that are read in groups of G.
inline int32_t room_of(const NormArgs& a, bool y_read, int G) {
  int room = rows_of_room(a.ldx, G);
  if (a.r) room = std::max(room, rows_of_room(a.ldr, G));
  if (y_read) room = std::max(room, rows_of_room(a.ldy, G));
  return room;
}

// How rows are taken in groups, if they can be.
struct Plan {
  int elements = 0;            // of a thread; 0: any layout
  int lanes = 0, threads = 0, stages = 0;
  bool split = false, ends = false;
  unsigned grid = 0;
  size_t smem = 0;
};

template <typename T>
bool same_phase(const void* p, int64_t ld, int64_t rows, int G, int64_t phase, int64_t shift) {
  if (!p) return true;
  return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / sizeof(T) % G) == phase && (rows == 1 || ld % G == shift);
}

// bytes: of one element of all operands that are read; params: fp32 rows of parameters in shared memory;
// most: CTAs at most; resident: threads of a CTA and of an SM that the kernels' registers leave room for;
// split: elements of a lane up to which a row goes to a warp's lanes; wide: lanes of 16 elements from which on a
// thread takes 32; rows: that a team takes at a time.
template <typename X, typename S, typename Y>
Plan make_plan(const NormArgs& a, size_t bytes, int params, int64_t most, int resident, int split, int wide, int rows = 1) {
  Plan p;
  constexpr int G = kGroup<X, S, Y>;
  const int64_t phase = reinterpret_cast<uintptr_t>(a.x) / sizeof(X) % G, shift = a.T > 1 ? a.ldx % G : 0;
  if (!same_phase<S>(a.r, a.ldr, a.T, G, phase, shift) || !same_phase<S>(a.s, a.lds, a.T, G, phase, shift) ||
      !same_phase<Y>(a.y, a.ldy, a.T, G, phase, shift))
    return p;
  const int groups = static_cast<int>((a.d + (shift ? G - 1 : phase) + G - 1) / G);   // of any row
  const int64_t sms = device_sm_count();
  auto lanes_of = [&](int elements) { return (groups + elements / G - 1) / (elements / G); };
  p.split = lanes_of(split) <= 32;
  p.ends = phase || shift || a.d % G;
  int E, teams;
  if (p.split) {
    E = lanes_of(8) <= 32 ? 8 : lanes_of(16) <= 32 ? 16 : 32;
    p.lanes = 32;
    while (p.lanes / 2 >= lanes_of(E)) p.lanes /= 2;
    teams = 256 / p.lanes;
    if (E == 32) resident = 512;
  } else {
    E = lanes_of(16) < wide ? 16 : 32;
    p.lanes = (lanes_of(E) + 31) / 32 * 32;
    if (p.lanes > (E == 32 ? 512 : 1024)) return p;
    if (E == 32) resident = 512;
    // rows for every SM before several for one
    teams = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kMaxTeams, resident / p.lanes, (a.T + sms - 1) / sms})));
  }
  // as many CTAs to an SM as their registers let in, fewer teams or CTAs where the rings would be too short
  int per_sm = std::max(1, resident / (teams * p.lanes));
  const size_t fixed = static_cast<size_t>(p.lanes) * E * 4 * params, stage = static_cast<size_t>(p.lanes) * E * bytes * rows;
  auto need = [&] { return per_sm * (fixed + static_cast<size_t>(teams) * p.stages * stage + kStaticSmem + 2 * 1024); };
  // stages: up to four, no more than a team has turns
  const int64_t turns = (a.T + per_sm * sms * teams * rows - 1) / (per_sm * sms * teams * rows);
  const int ahead = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, turns)));
  for (;;) {
    for (p.stages = ahead; p.stages > 2 && need() > kSharedPerSm;) --p.stages;
    if (need() <= kSharedPerSm) break;
    if (per_sm > 1) {
      --per_sm;
    } else if (teams > 1 && !p.split) {
      --teams;
    } else {      // one row at a time, or none
      p.stages = 1;
      if (need() > kSharedPerSm) return p;
      break;
    }
  }
  p.threads = teams * p.lanes;
  p.smem = fixed + static_cast<size_t>(teams) * p.stages * stage;
  p.elements = E;
  int64_t ctas = std::min({(a.T + teams - 1) / teams, most, per_sm * sms});
  if (shift) ctas = std::max<int64_t>(8, ctas / 8 * 8);
  p.grid = static_cast<unsigned>(ctas);
  return p;
}

// A kernel's limit of dynamic shared memory, raised where the plan's and the kernel's own arrays may together be more
// than every kernel has without asking.
template <typename F>
cudaError_t allow_smem(F f, size_t bytes) {
  return bytes + kStaticSmem > kDefaultSmem ? set_smem_once(reinterpret_cast<const void*>(f), bytes) : cudaSuccess;
}

}  // namespace moe
