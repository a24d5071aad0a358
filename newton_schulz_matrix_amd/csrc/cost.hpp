// cost.hpp - estimated times of the streamed products (stream.hpp), by which
// the entry points choose tiles and splits.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "xent.hpp"

namespace {

using namespace nsk;
using namespace nsr;

// Estimated time of a product in us: rounds of tiles over the compute units,
// each of so many us per k-tile and a fixed part, as measured on MI355X with
// random operands.
// (Two or three of the smallest float tiles on a compute unit, with stages of
// 16 KB, gained 5 to 10 % where tiles filled them evenly and lost up to 30 %
// where they did not: 300 x 1000 x 8191 took 76 and 56 us against 59.)
struct EdgeCost {
  int edge;
  double ktile, fixed;
};
constexpr EdgeCost kXentCost16[2] = {{kXentLarge<_Float16>, 0.90, 3.0}, {kXentSmall<_Float16>, 0.52, 2.0}};
constexpr EdgeCost kXentCost32[2] = {{kXentLarge<float>, 2.10, 2.5}, {kXentSmall<float>, 0.53, 1.5}};
// k-tiles go in groups of three (stream.hpp).
double tile_us(const EdgeCost& c, double ktiles) { return ceil(ktiles / 3) * 3 * c.ktile + c.fixed; }
double product_us(const EdgeCost& c, int64_t tiles, double ktiles) {
  return (double)((tiles + kXentGroups - 1) / kXentGroups) * tile_us(c, ktiles);
}
const EdgeCost* edge_costs(int es) { return es == 2 ? kXentCost16 : kXentCost32; }

// The gradients' two products in one launch: dW's tiles go round the
// work-groups, so that some have one more than the others; those others take
// part in `extra` rounds of dH's tiles before all do.  The number of rounds
// that ends first.
struct GradRounds {
  int extra = 0;
  double us = 1e300;
};
GradRounds grad_rounds(const EdgeCost& c, int64_t dw_tiles, double dw_ktiles, int64_t dh_tiles, double dh_ktiles) {
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(kXentGroups, dw_tiles + dh_tiles));
  const int64_t busy = dw_tiles % grid, idle = grid - busy;
  const double one_w = tile_us(c, dw_ktiles), one_h = tile_us(c, dh_ktiles);
  const double before = (double)(dw_tiles / grid) * one_w;
  GradRounds best;
  for (int64_t e = 0; e == 0 || (busy && e <= one_w / one_h + 1 && (e - 1) * idle < dh_tiles); ++e) {
    if (before + e * one_h >= best.us) break;
    const int64_t left = std::max<int64_t>(0, dh_tiles - e * idle), r = (left + grid - 1) / grid;
    const double us = before + std::max(busy ? one_w + r * one_h : 0, (e + r) * one_h);
    if (us < best.us) best = {(int)e, us};
  }
  return best;
}

// dH's splits to choose from: few rows leave most compute units without a
// tile of dH (35 x 434 x 84115: 4 tiles of 1315 k-tiles, 140 us with 8 splits).
constexpr int kXentSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32, 48, 64};

}  // namespace
