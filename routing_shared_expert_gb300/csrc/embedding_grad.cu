// Gradient of the token embedding's table: dtable_v = scale sum_{t: id_t = v} dout_t, in fp32 and in a fixed
// order, zeros (or what was there) for rows without a token.
//
// The tokens are sorted by their row, stably, so that a row's tokens are neighbours in ascending order.
// The sorted list is cut into chunks of 32 tokens (8, where they are few): a warp adds a chunk's gradients up over a
// slice of columns, run by run, and writes the rows whose run lies within the chunk.  A run over a chunk's end (a
// frequent token) leaves partial sums, which a second launch adds in the chunks' order.  The rows without a token get
// their zeros from other CTAs of the sort's and the join's launches, which leave HBM idle, and of the sums'.
// 32768 tokens to a fp32 table of 65536 x 2560: 136 us, 6.2 TB/s (the bytes at the copy rate 124 us): marks, counts and
// two sort passes about 20 us, half of it covered by zeros, sums 90 us at 83 % of the DRAM peak, join 10 us.  Small or
// narrow tables are bound by the five to six launches (4000 tokens to 1000 x 64: 20 us).
#include "embedding.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------------ zeros --

constexpr int kMaxZeroRows = 128;   // of a CTA that writes zeros

// Which rows of the table have no token: from a mark per row, or (few tokens) from the token numbers themselves.
struct Zeros {
  const uint8_t* has;      // [V], 1 for rows with a token
  void* table;
  int64_t ldt, V;
  int64_t from;            // first row of this launch's share, a multiple of eight
  unsigned ctas;           // CTAs that write it
  int32_t rows;            // of each, a multiple of eight
  int32_t d, bf16;
};

// Zeros for row v by one warp.
__device__ __forceinline__ void zero_row(const Zeros& z, int64_t v) {
  const int lane = threadIdx.x & 31;
  const int64_t size = z.bf16 ? 2 : 4, bytes = z.d * size;
  char* p = static_cast<char*>(z.table) + v * z.ldt * size;
  // whole 16-byte pieces, and what lies before and behind them element by element
  const int64_t head = min(bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(p) & 15)), body = (bytes - head) & ~int64_t{15};
  for (int64_t c = head + 16 * lane; c < head + body; c += 512) *reinterpret_cast<uint4*>(p + c) = make_uint4(0u, 0u, 0u, 0u);
  const int64_t at = lane < 16 ? lane * size : head + body + (lane - 16) * size;
  if (at < (lane < 16 ? head : bytes)) {
    if (z.bf16) *reinterpret_cast<uint16_t*>(p + at) = 0;
    else *reinterpret_cast<uint32_t*>(p + at) = 0u;
  }
}

// The zeros of the rows of one CTA of a share.
__device__ __forceinline__ void zeros_by_marks(const Zeros& z, unsigned cta) {
  const int64_t v0 = z.from + static_cast<int64_t>(cta) * z.rows, v1 = min(z.V, v0 + z.rows);
  for (int64_t v = v0 + (threadIdx.x >> 5); v < v1; v += blockDim.x >> 5)
    if (!z.has[v]) zero_row(z, v);
}
template <typename I>
__device__ __forceinline__ void zeros_by_tokens(const Zeros& z, unsigned cta, const I* ids, int T) {
  __shared__ uint32_t seen[kMaxZeroRows / 32];
  const int64_t v0 = z.from + static_cast<int64_t>(cta) * z.rows, v1 = min(z.V, v0 + z.rows);
  if (threadIdx.x < kMaxZeroRows / 32) seen[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < T; i += blockDim.x) {
    const int64_t r = static_cast<int64_t>(ids[i]) - v0;
    if (r >= 0 && r < z.rows) atomicOr(seen + (r >> 5), 1u << (r & 31));
  }
  __syncthreads();
  for (int64_t v = v0 + (threadIdx.x >> 5); v < v1; v += blockDim.x >> 5)
    if (!(seen[(v - v0) >> 5] >> ((v - v0) & 31) & 1)) zero_row(z, v);
}

__global__ void __launch_bounds__(256) clear_marks_kernel(uint4* has, int64_t n) {
  launch_dependents();
  wait_for_previous();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    has[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------------- sort --
// Radix sort by digits of up to nine bits from the lowest, each pass stable.  A tile is the tokens of one CTA.  Nine bits
// let every row number below 2^18 do with two passes, and a thread of the CTA own each digit.

constexpr int kDigits = 512, kSortThreads = 512, kSortWarps = kSortThreads / 32, kItems = 4;
constexpr int kTile = kSortThreads * kItems;      // tokens at a time
constexpr int kMaxTiles = 64;

struct SortArgs {
  const void* ids;
  int64_t V;
  int32_t T;
  int32_t tile;           // tokens of a CTA, a multiple of kTile
  int32_t tiles;
  int32_t shift, bits;    // of this pass's digit
  int32_t next_shift, next_bits;   // of the next pass's, 0 bits after the last
  const int2* in;         // (row, token) of earlier passes; NULL: the token numbers
  int2* out;
  int32_t* hist;          // [tiles][kDigits] tokens of each digit in each tile of `in`
  int32_t* next_hist;     // the same of `out`, zero at the launch
  int32_t* status;
  uint8_t* has;           // marks to set, or NULL
  Zeros zeros;            // what CTAs past the tiles write
};

template <typename I>
__device__ __forceinline__ int2 sort_item(const SortArgs& a, int i, int32_t* status) {
  if (a.in) return a.in[i];
  const int64_t v = token_row(static_cast<const I*>(a.ids), i, a.V, status);
  return make_int2(static_cast<int>(v < 0 ? a.V : v), i);      // no token: behind the last row
}

// Digits of each tile, and zeros for the counts of the next pass.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ int32_t n[kDigits];
  __shared__ int32_t marked[2048];      // rows that this CTA has marked lately: a frequent one's mark is not stored at each token
  launch_dependents();
  wait_for_previous();
  n[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < 2048; i += kSortThreads) marked[i] = -1;
  if (a.next_bits) a.next_hist[blockIdx.x * kDigits + threadIdx.x] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
  for (int i = t0 + threadIdx.x; i < t1; i += kSortThreads) {
    const int v = sort_item<I>(a, i, a.status).x;
    atomicAdd(n + (v >> a.shift & ((1 << a.bits) - 1)), 1);
    if (a.has && v < a.V && marked[v & 2047] != v) {
      marked[v & 2047] = v;
      a.has[v] = 1;
    }
  }
  __syncthreads();
  a.hist[blockIdx.x * kDigits + threadIdx.x] = n[threadIdx.x];
}

// The sum of v over the threads before this one.
__device__ __forceinline__ int exclusive_scan(int v, int32_t* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int w = lane < kSortWarps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < kSortWarps; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return s - v + (warp > 0 ? before : 0);
}

// Where the items of up to kTile neighbours go: item j of a thread is number warp * 128 + 32 j + lane.  `base` holds
// where each digit's next item goes and is moved on; NULL: these are all items, and the ranking's own counts say it.
using WarpCounts = int32_t (&)[kSortWarps][kDigits];
__device__ __forceinline__ void place_items(WarpCounts warp_n, int32_t* base, int32_t* part, const int (&digit)[kItems],
                                            const bool (&on)[kItems], int (&to)[kItems]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = lane; i < kDigits; i += 32) warp_n[warp][i] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const unsigned peers = __match_any_sync(0xffffffffu, on[j] ? digit[j] : -1 - lane);
    const int before = on[j] ? warp_n[warp][digit[j]] : 0;
    to[j] = before + __popc(peers & ((1u << lane) - 1));
    __syncwarp();
    if (on[j] && (peers & ((1u << lane) - 1)) == 0) warp_n[warp][digit[j]] = before + __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  int at;
  if (base) {
    at = base[threadIdx.x];
  } else {
    int all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) all += warp_n[w][threadIdx.x];
    at = exclusive_scan(all, part);
  }
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const int n = warp_n[w][threadIdx.x];
    warp_n[w][threadIdx.x] = at;
    at += n;
  }
  if (base) base[threadIdx.x] = at;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kItems; ++j)
    if (on[j]) to[j] += warp_n[warp][digit[j]];
  __syncthreads();
}

template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(SortArgs a) {
  __shared__ int32_t warp_n[kSortWarps][kDigits], base[kDigits], part[kSortWarps];
  launch_dependents();
  wait_for_previous();
  if (blockIdx.x >= static_cast<unsigned>(a.tiles)) {
    zeros_by_marks(a.zeros, blockIdx.x - a.tiles);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this tile's share of each digit begins behind the lower digits and the earlier tiles
  int before = 0, all = 0;
#pragma unroll 16
  for (int t = 0; t < a.tiles; ++t) {
    const int n = a.hist[t * kDigits + threadIdx.x];
    if (t < static_cast<int>(blockIdx.x)) before += n;
    all += n;
  }
  const int lower = exclusive_scan(all, part);
  base[threadIdx.x] = lower + before;
  const int t0 = blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
  for (int i0 = t0; i0 < t1; i0 += kTile) {
    int2 item[kItems];
    int digit[kItems], to[kItems];
    bool on[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int i = i0 + warp * 32 * kItems + 32 * j + lane;
      on[j] = i < t1;
      item[j] = on[j] ? sort_item<I>(a, i, nullptr) : make_int2(0, 0);
      digit[j] = item[j].x >> a.shift & ((1 << a.bits) - 1);
    }
    __syncthreads();
    place_items(warp_n, base, part, digit, on, to);
#pragma unroll
    for (int j = 0; j < kItems; ++j)
      if (on[j] && to[j] < a.T) {      // token numbers that change under the call stay within the list
        a.out[to[j]] = item[j];
        if (a.next_bits)
          atomicAdd(a.next_hist + to[j] / a.tile * kDigits + (item[j].x >> a.next_shift & ((1 << a.next_bits) - 1)), 1);
      }
  }
}

// All passes for at most kTile tokens, in the first CTA's shared memory; the others write all zeros.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(SortArgs a) {
  __shared__ alignas(16) int32_t warp_n[kSortWarps][kDigits];
  __shared__ int32_t part[kSortWarps];
  static_assert(sizeof(warp_n) >= kTile * sizeof(int2), "the counts' place holds the list between passes");
  int2* list = reinterpret_cast<int2*>(warp_n);
  launch_dependents();
  wait_for_previous();
  if (blockIdx.x > 0) {
    zeros_by_tokens(a.zeros, blockIdx.x - 1, static_cast<const I*>(a.ids), a.T);
    return;
  }
  const int i0 = (threadIdx.x >> 5) * 32 * kItems + (threadIdx.x & 31);
  int2 item[kItems];
  int digit[kItems], to[kItems];
  bool on[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    on[j] = i0 + 32 * j < a.T;
    item[j] = on[j] ? sort_item<I>(a, i0 + 32 * j, a.status) : make_int2(0, 0);
  }
  for (int shift = 0; shift < a.bits; shift += 9) {      // bits: of a whole row number
#pragma unroll
    for (int j = 0; j < kItems; ++j) digit[j] = item[j].x >> shift & (kDigits - 1);
    place_items(warp_n, nullptr, part, digit, on, to);
#pragma unroll
    for (int j = 0; j < kItems; ++j)
      if (on[j]) list[to[j]] = item[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kItems; ++j)
      if (on[j]) item[j] = list[i0 + 32 * j];
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j)
    if (on[j]) a.out[i0 + 32 * j] = item[j];
}

// ------------------------------------------------------------------------- sums --

struct SumArgs {
  EmbedArgs e;
  const int2* list;        // (row, token), sorted; row V behind the last: no token
  float* partial;          // [chunks][2][d]: of the run that enters a chunk, of the one that leaves it
  int32_t T, chunk, chunks, slices;      // tokens; of a warp, 8 or 32; how many of those; parts of a row
  unsigned sum_ctas;       // of the launch; those behind them write zeros
  Zeros zeros;
};

// One slice of a table row: v times the scale, or added to what the row holds.
template <typename W, bool ALIGNED>
__device__ __forceinline__ void write_row(const EmbedArgs& a, int64_t row, int c0, const float2 (&v)[4]) {
  W* p = static_cast<W*>(a.dst) + row * a.ldt;
  float2 u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = mul2(v[j], both(a.scale));
  if (a.accumulate) {
    Slice<W, ALIGNED> held;
    float2 h[4];
    held.load(p, c0, a.d);
    held.unpack(h);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = add2(h[j], u[j]);
  }
  store_slice<W, ALIGNED>(p, c0, a.d, u);
}

template <typename Y, typename W, bool ALIGNED>
__device__ __forceinline__ void sum_chunk(const SumArgs& s, int chunk, int c0) {
  const EmbedArgs& a = s.e;
  const int lane = threadIdx.x & 31;
  const int i0 = chunk * s.chunk, n = min(s.chunk, s.T - i0);
  int2 mine = lane < n ? s.list[i0 + lane] : make_int2(static_cast<int>(a.V), 0);
  if (mine.x < 0 || static_cast<unsigned>(mine.y) >= static_cast<unsigned>(s.T)) mine = make_int2(static_cast<int>(a.V), 0);
  const int entering = i0 > 0 ? s.list[i0 - 1].x : -1, leaving = i0 + n < s.T ? s.list[i0 + n].x : -1;
  float* const partial = s.partial + static_cast<int64_t>(chunk) * 2 * a.d;
  float2 acc[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
  bool first = true;       // of the chunk's runs
  int row = __shfl_sync(0xffffffffu, mine.x, 0);
  constexpr int kAhead = 8;      // tokens on their way
  for (int b = 0; b < s.chunk && row < a.V; b += kAhead) {
    Slice<Y, ALIGNED> w[kAhead];
    int rows[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      rows[j] = __shfl_sync(0xffffffffu, mine.x, b + j);
      const int t = __shfl_sync(0xffffffffu, mine.y, b + j);
      if (rows[j] < a.V) w[j].load(static_cast<const Y*>(a.src) + t * a.ldo, c0, a.d);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (rows[j] != row) {        // the run ends before this token
        if (first && row == entering) store_slice<float, ALIGNED>(partial, c0, a.d, acc);
        else write_row<W, ALIGNED>(a, row, c0, acc);
        first = false;
        row = rows[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = both(0.f);
      }
      if (row >= a.V) break;
      float2 v[4];
      w[j].unpack(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = add2(acc[i], v[i]);
    }
  }
  if (row >= a.V) return;
  const bool enters = first && row == entering;
  if (enters || row == leaving) store_slice<float, ALIGNED>(partial + (enters ? 0 : a.d), c0, a.d, acc);
  else write_row<W, ALIGNED>(a, row, c0, acc);
}

template <typename Y, typename W, bool ALIGNED>
__global__ void __launch_bounds__(256, 2) embed_sum_kernel(SumArgs s) {
  launch_dependents();
  wait_for_previous();
  if (blockIdx.x >= s.sum_ctas) {
    zeros_by_marks(s.zeros, blockIdx.x - s.sum_ctas);
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int chunk = static_cast<int>(item / s.slices);
  if (chunk >= s.chunks) return;
  sum_chunk<Y, W, ALIGNED>(s, chunk, static_cast<int>(item - static_cast<int64_t>(chunk) * s.slices) * kColumns);
}

// Partial sums of chunks [b0, b1) of the run that begins in chunk `from`, in order.
template <bool ALIGNED>
__device__ __forceinline__ void add_partials(const SumArgs& s, int from, int b0, int b1, int c0, float2 (&acc)[4]) {
  const int d = s.e.d;
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = both(0.f);
  constexpr int kAhead = 8;
  for (int b = b0; b < b1; b += kAhead) {
    Slice<float, ALIGNED> w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (b + k < b1) w[k].load(s.partial + (static_cast<int64_t>(b + k) * 2 + (b + k == from ? 1 : 0)) * d, c0, d);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (b + k < b1) {
        float2 u[4];
        w[k].unpack(u);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = add2(acc[j], u[j]);
      }
  }
}

// Runs over several chunks: the sum of the chunk that a run begins in and of those that it enters, in order.  A warp
// looks whether a run begins in its chunk and goes on, and adds runs of up to kAlone chunks up by itself; longer
// ones are cut into eight stretches for the CTA's warps.
constexpr int kAlone = 32;

template <typename W, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_join_kernel(SumArgs s) {
  __shared__ float2 part[8][4][32];
  __shared__ int long_row[8], long_end[8];
  wait_for_previous();
  const unsigned groups = (s.chunks + 7) / 8;
  if (blockIdx.x >= groups * s.slices) {
    zeros_by_marks(s.zeros, blockIdx.x - groups * s.slices);
    return;
  }
  const EmbedArgs& a = s.e;
  const int group = blockIdx.x % groups, slice = blockIdx.x / groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = slice * kColumns;
  const int chunk = group * 8 + warp, first = chunk * s.chunk, next = first + s.chunk;
  int row = -1, end = 0;           // the run's row, and the chunk behind the last that it enters
  if (next < s.T) {
    const int before = first > 0 ? s.list[first - 1].x : -1, head = s.list[first].x, tail = s.list[next - 1].x,
              after = s.list[next].x;
    if (tail < a.V && after == tail && (before != tail || head != tail)) row = tail;
  }
  if (row >= 0) {
    for (end = chunk + 1;; end += 32) {      // 32 chunks at a time: the last item of each that the run fills
      const int at = min((end + lane) * s.chunk + s.chunk, s.T) - 1;
      const unsigned fills = __ballot_sync(0xffffffffu, end + lane < s.chunks && s.list[at].x == row);
      if (fills != 0xffffffffu) {
        end += __popc(fills);
        break;
      }
    }
    if (end < s.chunks && s.list[end * s.chunk].x == row) ++end;      // it ends within this one
  }
  const bool alone = row >= 0 && end - chunk <= kAlone;
  if (lane == 0) {
    long_row[warp] = row >= 0 && !alone ? row : -1;
    long_end[warp] = end;
  }
  float2 acc[4];
  if (alone) {
    add_partials<ALIGNED>(s, chunk, chunk, end, c0, acc);
    write_row<W, ALIGNED>(a, row, c0, acc);
  }
  __syncthreads();
  for (int k = 0; k < 8; ++k) {
    if (long_row[k] < 0) continue;
    const int from = group * 8 + k, to = long_end[k], per = (to - from + 7) / 8, b0 = from + warp * per;
    add_partials<ALIGNED>(s, from, min(b0, to), min(to, b0 + per), c0, acc);
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][j][lane] = acc[j];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int w = 1; w < 8; ++w) acc[j] = add2(acc[j], part[w][j][lane]);
      write_row<W, ALIGNED>(a, long_row[k], c0, acc);
    }
    __syncthreads();
  }
}

// Gradient without a sort: a CTA owns kScanRows rows of the table and 256 columns, reads every
// token number, keeps those of its rows in order, and adds their gradients up in shared memory,
// a thread per column.
constexpr int kScanRows = 32, kScanIds = 8 * 256;

template <typename I, typename Y, typename W>
__global__ void __launch_bounds__(256) embed_scan_kernel(EmbedArgs a) {
  launch_dependents();
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
  wait_for_previous();
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
      for (int i0 = 0; i0 < total; i0 += 8) {      // eight loads on their way
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = i0 + i < total ? to_f32(static_cast<const Y*>(a.src)[list_t[i0 + i] * a.ldo + c]) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < total) acc[list_v[i0 + i]][tid] += v[i];
      }
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

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

int bits_of(int64_t v) {
  int b = 1;
  while (v >> b) ++b;
  return b;
}

// Whether every block of the table's rows looks through the tokens, instead of their being sorted: while they are so
// few that one CTA can add a frequent one up, and all CTAs together read few token numbers (300 tokens to
// 1000 x 256: 6.2 us; 2000 tokens to 500 x 1024 45 us, sorted 12).
bool scans(int64_t T, int64_t V, int32_t d) {
  const int64_t ctas = (V + kScanRows - 1) / kScanRows * ((d + 255) / 256);
  return T <= 512 && T * ctas <= (1 << 20);
}

// Tokens of a warp.  Few tokens leave most of the GPU empty, and a warp that takes them one batch of loads after another
// is what the launch waits for: 1200 tokens of 450 24 us with 8, 54 with 32; 9600 of 1024 30 and 35.  With the GPU
// full the partial sums' traffic counts: 65536 of 64 37 and 31; 19200 of 4096 100 and 85.
constexpr int kChunk = 32, kFewChunk = 8;
constexpr int64_t kFewSlices = 152 * 2 * 16 * kFewChunk;      // tokens x slices of a row: twice the warps that are resident
// A row with most of the tokens has a partial sum per chunk, and one CTA adds them up: 32768 tokens of one row 88 us with 8,
// 42 with 32, while 19200 spread ones gain only 10 %.
constexpr int64_t kFewTokens = 16384;

struct GradLayout {
  bool scan;
  int32_t tiles, tile, chunk, chunks;
  size_t list[2], hist[2], has, partial, total;
};
GradLayout grad_layout(int64_t T, int64_t V, int32_t d) {
  GradLayout l{};
  l.scan = T == 0 || scans(T, V, d);
  if (l.scan) return l;
  const int64_t per = (T + kMaxTiles - 1) / kMaxTiles;
  l.tile = static_cast<int32_t>((per + kTile - 1) / kTile * kTile);
  l.tiles = static_cast<int32_t>((T + l.tile - 1) / l.tile);
  const int64_t few = std::min(kFewTokens, kFewSlices / ((d + kColumns - 1) / kColumns));
  l.chunk = T <= few ? kFewChunk : kChunk;
  l.chunks = static_cast<int32_t>((T + l.chunk - 1) / l.chunk);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    l.list[i] = take(static_cast<size_t>(T) * 8);
    // for as many tiles as any smaller T has, so that its workspace does for all of those
    l.hist[i] = take(static_cast<size_t>(std::min<int64_t>(kMaxTiles, (T + kTile - 1) / kTile)) * kDigits * 4);
  }
  l.has = take(static_cast<size_t>(V + 15) / 16 * 16);
  // what any smaller T wants, too
  const int64_t most = std::max((T + kChunk - 1) / kChunk, (std::min(T, few) + kFewChunk - 1) / kFewChunk);
  l.partial = take(static_cast<size_t>(most) * 2 * static_cast<size_t>(d) * 4);
  l.total = o;
  return l;
}

// Bytes of zeros beside one pass of the sort, and beside the join: about what HBM takes during it.
constexpr int64_t kZerosBeside = 48 << 20;
int64_t rows_beside(const Zeros& z) { return kZerosBeside / (static_cast<int64_t>(z.d) * (z.bf16 ? 2 : 4)) + 1; }

// The next share of the table's rows for the CTAs of one launch, `rows` at most.
Zeros next_zeros(Zeros& z, int64_t rows) {
  Zeros part = z;
  const int64_t left = (z.V - z.from + z.rows - 1) / z.rows;
  part.ctas = static_cast<unsigned>(std::max<int64_t>(0, std::min(left, (rows + z.rows - 1) / z.rows)));
  z.from += part.ctas * static_cast<int64_t>(z.rows);
  return part;
}

// The sorted list of (row, token); zeros: of what is left when the sort is done.
template <typename I>
cudaError_t sort_tokens(const EmbedArgs& a, const GradLayout& l, const int2** list, Zeros& zeros, cudaStream_t s) {
  SortArgs p{};
  p.ids = a.ids;
  p.V = a.V;
  p.T = static_cast<int32_t>(a.T);
  p.tile = l.tile;
  p.tiles = l.tiles;
  p.status = a.status;
  const int bits = bits_of(a.V);
  int2* lists[2] = {reinterpret_cast<int2*>(a.scratch + l.list[0]), reinterpret_cast<int2*>(a.scratch + l.list[1])};
  int32_t* hists[2] = {reinterpret_cast<int32_t*>(a.scratch + l.hist[0]), reinterpret_cast<int32_t*>(a.scratch + l.hist[1])};
  if (a.T <= kTile) {
    p.bits = bits;
    p.out = lists[0];
    p.zeros = next_zeros(zeros, a.V);
    *list = lists[0];
    return launch_over(sort_small_kernel<I>, dim3(1 + p.zeros.ctas), kSortThreads, 0, s, p);
  }
  cudaError_t e = cudaSuccess;
  if (zeros.from < a.V) {
    const int64_t pieces = (a.V + 15) / 16;
    p.has = reinterpret_cast<uint8_t*>(a.scratch + l.has);
    e = launch_over(clear_marks_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(1024, (pieces + 255) / 256))), 256, 0, s,
                    reinterpret_cast<uint4*>(p.has), pieces);
  }
  const int passes = (bits + 8) / 9, width = (bits + passes - 1) / passes;
  for (int k = 0; k < passes && e == cudaSuccess; ++k) {
    p.shift = k * width;
    p.bits = std::min(width, bits - p.shift);
    p.next_shift = p.shift + width;
    // the counts of the second pass are kept by the first, those of later ones are taken anew
    p.next_bits = k == 0 && passes > 1 ? std::min(width, bits - p.next_shift) : 0;
    p.in = k ? lists[(k - 1) % 2] : nullptr;
    p.out = lists[k % 2];
    p.hist = hists[k % 2];
    p.next_hist = hists[(k + 1) % 2];
    if (k != 1) e = launch_over(sort_count_kernel<I>, dim3(static_cast<unsigned>(l.tiles)), kSortThreads, 0, s, p);
    p.has = nullptr;
    p.zeros = next_zeros(zeros, rows_beside(zeros));
    if (e == cudaSuccess)
      e = launch_over(sort_pass_kernel<I>, dim3(static_cast<unsigned>(l.tiles) + p.zeros.ctas), kSortThreads, 0, s, p);
    *list = p.out;
  }
  return e;
}

template <typename Y, typename W, bool ALIGNED>
cudaError_t launch_sums(SumArgs p, const Zeros& beside_join, cudaStream_t s) {
  const cudaError_t e = launch_over(embed_sum_kernel<Y, W, ALIGNED>, dim3(p.sum_ctas + p.zeros.ctas), 256, 0, s, p);
  if (e != cudaSuccess || p.chunks < 2) return e;
  p.zeros = beside_join;
  const unsigned ctas = static_cast<unsigned>((p.chunks + 7) / 8) * static_cast<unsigned>(p.slices);
  return launch_over(embed_join_kernel<W, ALIGNED>, dim3(ctas + p.zeros.ctas), 256, 0, s, p);
}

template <typename I, typename Y, typename W>
cudaError_t launch_grad(const EmbedArgs& a, cudaStream_t s) {
  const GradLayout l = grad_layout(a.T, a.V, a.d);
  if (l.scan) {
    const dim3 grid(static_cast<unsigned>((a.V + kScanRows - 1) / kScanRows), static_cast<unsigned>((a.d + 255) / 256));
    return launch_over(embed_scan_kernel<I, Y, W>, grid, 256, 0, s, a);
  }
  SumArgs p{};
  Zeros zeros{};
  zeros.has = reinterpret_cast<const uint8_t*>(a.scratch + l.has);
  zeros.table = a.dst;
  zeros.ldt = a.ldt;
  zeros.V = a.V;
  zeros.from = a.accumulate ? a.V : 0;
  zeros.d = a.d;
  zeros.bf16 = sizeof(W) == 2;
  // a CTA's rows: about 64 KB of them, so that a share spreads over the SMs; at least one for each of its warps
  zeros.rows = static_cast<int32_t>(std::min<int64_t>(kMaxZeroRows, std::max<int64_t>(8, (64 << 10) / (static_cast<int64_t>(a.d) * sizeof(W)) / 8 * 8)));
  const cudaError_t e = sort_tokens<I>(a, l, &p.list, zeros, s);
  if (e != cudaSuccess) return e;
  // what is left: a share for the join, when it is launched, and the rest beside the sums
  const int64_t left = a.V - zeros.from, late = l.chunks > 1 ? std::min(left, rows_beside(zeros)) : 0;
  p.zeros = next_zeros(zeros, left - late);
  const Zeros beside_join = next_zeros(zeros, a.V);
  p.e = a;
  p.partial = reinterpret_cast<float*>(a.scratch + l.partial);
  p.T = static_cast<int32_t>(a.T);
  p.chunk = l.chunk;
  p.chunks = l.chunks;
  p.slices = (a.d + kColumns - 1) / kColumns;
  p.sum_ctas = static_cast<unsigned>((static_cast<int64_t>(p.chunks) * p.slices + 7) / 8);
  return groups_of_eight<Y>(a.src, a.ldo, a.d) && groups_of_eight<W>(a.dst, a.ldt, a.d) ? launch_sums<Y, W, true>(p, beside_join, s)
                                                                                        : launch_sums<Y, W, false>(p, beside_join, s);
}
template <typename I, typename Y>
cudaError_t launch_table(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.table_dtype == MOE_F32 ? launch_grad<I, Y, float>(a, s) : launch_grad<I, Y, __nv_bfloat16>(a, s);
}
template <typename I>
cudaError_t launch_out(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.out_dtype == MOE_F32 ? launch_table<I, float>(a, c, s) : launch_table<I, __nv_bfloat16>(a, c, s);
}

}  // namespace

size_t embedding_scratch(int64_t T, int64_t V, int32_t d) { return grad_layout(T, V, d).total; }

cudaError_t launch_embedding_backward(const EmbedArgs& a, const moe_embedding_config& c, cudaStream_t s) {
  return c.ids_int64 ? launch_out<int64_t>(a, c, s) : launch_out<int32_t>(a, c, s);
}

}  // namespace moe
