// The rows and token tiles of an expert, from offsets that may break their rule.
// Plain C++, so that it can be checked on the host.
#pragma once

#include <cstdint>

namespace nm {

// Rows lo <= t < hi of an expert whose offsets are `first` and `next`.
constexpr int rows_lo(int32_t first, int T) { return first < 0 ? 0 : first < T ? first : T; }
constexpr int rows_hi(int32_t next, int lo, int T) { return next < lo ? lo : next < T ? next : T; }

// Tiles that T tokens of E experts can make: sum ceil(n_e / BT) with at most
// min(E, T) experts that have tokens.
constexpr int64_t group_max_tiles(int64_t T, int64_t E, int64_t BT) {
  return (T + (E < T ? E : T) * (BT - 1)) / BT;
}

// Sums of tile counts stop here: far above any tile's number (T <= 2^24, E < 2^16),
// and two of them still fit 31 bits, whatever rows the offsets give to how many experts.
constexpr int kTileSumMax = 1 << 29;
constexpr int tile_sum(int a, int b) { return a + b < kTileSumMax ? a + b : kTileSumMax; }

}  // namespace nm
