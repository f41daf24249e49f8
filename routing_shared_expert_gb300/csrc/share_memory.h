// Whether tensors of a list share memory (host only): exact for rows of any widths and strides.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <utility>
#include <vector>

namespace moe {

// What a tensor occupies: rows of `width` bytes, `pitch` apart (one row: 0), from lo up to hi.
struct Reach {
  uintptr_t lo, hi;
  uint64_t pitch, width;
  bool written;
};

inline Reach reach_of(const void* p, uint64_t rows, uint64_t width, uint64_t pitch, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (rows - 1) * pitch + width, rows > 1 ? pitch : 0, width, written};
}

// Sum over k = 0 .. n - 1 of floor((a k + b) / m), modulo 2^64, in as many steps as Euclid's algorithm takes for a and m:
// whole multiples of m are taken out, and the points under what is left are counted along the other axis.
inline uint64_t floor_sum(uint64_t n, uint64_t m, uint64_t a, uint64_t b) {
  using Wide = unsigned __int128;
  uint64_t sum = 0;
  for (;;) {
    sum += static_cast<uint64_t>(Wide{n} * (n - 1) / 2) * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const Wide top = Wide{a} * n + b;
    if (top < m) return sum;
    n = static_cast<uint64_t>(top / m);
    b = static_cast<uint64_t>(top % m);
    std::swap(a, m);
  }
}

// A row of a from s on meets one of b's, which repeat every P bytes from b.lo on, where s + a.width - 1 - b.lo is at most
// a.width + b.width - 2 past a multiple of P.  Of a only the rows that reach into b's span count; one of those that met
// a row before b's first or behind its last would hold b's first or last byte too.
inline bool share_memory(Reach a, Reach b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (b.pitch == 0) std::swap(a, b);
  if (b.pitch == 0) return true;                             // one row each
  uint64_t first = 0, last = 0;
  if (a.pitch) {
    if (a.lo + a.width <= b.lo) first = (b.lo - a.lo - a.width) / a.pitch + 1;
    last = std::min((a.hi - a.lo - a.width) / a.pitch, (b.hi - 1 - a.lo) / a.pitch);
    if (first > last) return false;                          // b lies between two rows of a
  }
  const uint64_t P = b.pitch, reach = a.width + b.width - 2, from = a.lo + first * a.pitch + a.width - 1 - b.lo;
  if (reach >= P - 1) return true;
  if (first == last || a.pitch == P) return from % P <= reach;     // one row, or rows that all lie alike
  return floor_sum(last - first + 1, P, a.pitch, from + P) != floor_sum(last - first + 1, P, a.pitch, from + P - reach - 1);
}

// Whether one that is written shares memory with any other of the list, which is sorted.
inline bool any_written_is_shared(std::vector<Reach>& list) {
  std::sort(list.begin(), list.end(), [](const Reach& a, const Reach& b) { return a.lo < b.lo; });
  std::vector<Reach> open;
  for (const Reach& e : list) {
    size_t k = 0;
    for (const Reach& o : open) {
      if (o.hi <= e.lo) continue;
      if ((o.written || e.written) && share_memory(o, e)) return true;
      open[k++] = o;
    }
    open.resize(k);
    open.push_back(e);
  }
  return false;
}

}  // namespace moe
