// Which groups over a row's ends may be copied whole.
//
// A group of G elements that a row fills only in part reaches at most G - 1 elements past the row, into the gap to the
// next row and into that row, or likewise before it.  The copy stays within the tensor's span, from its first row's
// first element to its last row's last one, where the rows between the row and that end hold as much: one row, where
// rows are G - 1 elements apart or more, else G - 1 rows, since rows are one element apart at least.  The groups of the
// `room` rows at either end of the tensor are copied element by element.
#pragma once

#include <cstdint>

namespace moe {

constexpr int rows_of_room(int64_t ld, int G) { return ld >= G - 1 ? 1 : G - 1; }

// mask: the group's elements that lie in the row, at least one and not all of them.
constexpr bool copied_whole(int row, int T, int room, unsigned mask, int G) {
  return (row >= room || (mask & 1)) && (row < T - room || mask >> (G - 1));
}

}  // namespace moe
