// Ranges of the copies of ragged_fp8_tile.hip.  Plain C++, so that the host compiles the same arithmetic.
//
// A copy's lanes are checked as offset >= range - scalar offset.  The difference must not wrap: a scalar offset
// past the range would let lanes read what lies behind it.
#pragma once

#include <cstdint>

#include "both_sides.h"

namespace mx {

// Bytes of `rows` rows of `width` bytes, `pitch` apart; none for no rows (a tile's second run of 16 weight rows
// begins past the last one in a last tile of 16 columns and fewer).
MX_BOTH_SIDES int64_t rows_range(int64_t rows, int64_t pitch, int64_t width) {
  return rows <= 0 ? 0 : (rows - 1) * pitch + width;
}

// The scalar offset (within a row) beside such a range: 0 where it is empty.
MX_BOTH_SIDES uint32_t row_offset(uint32_t range, uint32_t offset) { return range == 0 ? 0u : offset; }

}  // namespace mx
