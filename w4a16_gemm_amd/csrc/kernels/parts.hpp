// How many parts of the contraction the tiles past whole rounds are split into (plan.hpp).
// The kernels that write partial sums and those that add them each work it out for themselves,
// so the rule is whole numbers alone: every compilation of it gives the same answer.
#pragma once

#include <cstdint>

namespace w4a16 {

// What a part more of `rest` tiles costs: 16 rest / outputs in the time of a tile.  Their
// partial sums are written and read.  (512 KB per tile of 256 rows and 8 XCDs' tiles at 5 TB/s, a step of 64
// outputs being 2.3 us, are 23 rest / outputs; less than that is measured.)
constexpr int kPartCost = 16;

// `rest` tiles, fewer than `side`, on `side` places that run at once, 32 or 64: the parts f, at
// most `most`, of the least rounds / f + f kPartCost rest / outputs, of equal ones the fewest, two
// rounds at most.  Where two workgroups share a compute unit (side 64), one alone takes 0.6 of
// their time: a round of up to 32 parts.  Costs are compared as fractions n / f, n in units of
// 1 / (5 outputs): below 2^28, since most is at most 32 and outputs at most 2^24.
constexpr int parts_of(int rest, int most, int side, int outputs) {
  if (rest <= 0) return 1;
  int best = 1;
  int64_t least = 0;
  for (int f = 1; f <= most && (f == 1 || f * rest <= 2 * side); ++f) {
    const int fifths = side == 64 && f * rest <= 32 ? 3 : f * rest <= side ? 5 : 10;
    const int64_t n = static_cast<int64_t>(outputs) * fifths + static_cast<int64_t>(5 * kPartCost) * rest * f * f;
    if (f == 1 || n * best < least * f) least = n, best = f;
  }
  return best;
}

}  // namespace w4a16
