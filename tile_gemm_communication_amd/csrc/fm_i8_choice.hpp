// fm_i8_choice.hpp -- which macro-tile an 8-bit product of many rows takes.
// Plain functions of sizes, for the host alone.
#pragma once

#include <stdint.h>

namespace fm {

constexpr int kI8Step = 128;   // bytes of k in a stage

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile of a product by what its rounds take: a K step of one block on a compute unit
// alone, of each of two there, and a tile's fixed part (us).  Fitted to 180 products of
// 65..8192 rows, 1024..12288 columns and as much k (the choice is 0.5% slower than the best
// of the seven on average; 64 x 64 tiles for all would be 26%, 256 x 256 for all 120%).  The
// small tiles take 0.2 us for the 16 KiB of a step with 32 tiles on the chip as with 192, with
// twice the stages or with a ring for each wave instead (loads alone reach 145 GB/s a unit, so
// it is not their path by itself); the large ones are bound by the matrix cores under the power
// limit.
struct TileChoice {
  int bm, bn, resident;
  double alone, shared, fixed;
};
constexpr TileChoice kTileChoices[] = {
    {64, 64, 2, 0.195, 0.397, 1.4},   {64, 128, 2, 0.267, 0.639, 2.1}, {128, 128, 1, 0.403, 0, 3.6},
    {128, 192, 1, 0.499, 0, 6.0},     {256, 128, 1, 0.631, 0, 5.7},    {256, 192, 1, 0.808, 0, 9.6},
    {256, 256, 1, 1.012, 0, 9.8},
};

inline int choose_tile(int64_t M, int64_t N, int64_t K, int cus) {
  const double steps = (double)ceil_div(K, kI8Step);
  int best = 0;
  double least = 0;
  for (int i = 0; i < (int)(sizeof(kTileChoices) / sizeof(kTileChoices[0])); ++i) {
    const TileChoice& c = kTileChoices[i];
    const int64_t each = ceil_div(ceil_div(M, c.bm) * ceil_div(N, c.bn), cus);
    const double one = steps * c.alone + c.fixed, two = steps * c.shared + c.fixed;
    const double time = c.resident == 1 ? each * one : each / 2 * two + each % 2 * one;
    if (i == 0 || time < least) {
      best = i;
      least = time;
    }
  }
  return best;
}

}  // namespace fm
