// fm_w4_index.hpp -- where the 4-bit products' loads of scales and zeros start.
// Plain integer functions, for host and device.
#pragma once

namespace fm {

// The column at which the loads of a block's 16-column tile start: n0 + tile, or n0 for
// a tile past N, whose values are not used.
constexpr int tile_column(int n0, int tile, int N) { return n0 + tile < N ? n0 + tile : n0; }

// Byte offset of `group` and `column` in one matrix's scales [groups, N] of 16 bits
// (of the zeros: half of it); groups past the last read the last.  It is the scalar
// part of a buffer load's offset.  some: 0 with no groups at all.
constexpr int scale_offset(int group, int groups, int column, int N, int some) {
  const int g = group < groups ? group : groups - 1;
  return (g * N + column) * 2 * some;
}

}  // namespace fm
