// Token tiles of rows ordered by expert: expert e owns rows offsets[e] ..
// offsets[e+1]-1 of T, and each expert's rows are cut into tiles of BT tokens of
// their own.  The offsets lie on the device, so the host knows only how many
// tiles there can be; which they are is found on the device, by every workgroup
// for itself (group_find: a few dependent loads, for kernels that are over in
// microseconds) or once for all by group_tiles_kernel (kernels whose workgroups
// walk many tiles).
//
// Offsets that do not ascend or leave [0, T] are clamped one by one
// (nm_offsets.h), so no access leaves the arrays, whatever they hold.
#pragma once

#include "nm_device.h"
#include "nm_offsets.h"

namespace nm {

// A tile's expert and its first token and the end of the expert's rows.
struct GroupTile {
  int e, t0, t1;
};

__device__ inline void group_range(const int32_t* __restrict__ offsets, int e, int T, int& lo, int& hi) {
  lo = rows_lo(offsets[e], T);
  hi = rows_hi(offsets[e + 1], lo, T);
}

// Tile number `tile` by the whole wave (64 experts at a time); false past the last.
// The results are the same in every lane and leave through readfirstlane: the
// compiler does not see that through the loop, and a descriptor made from what it
// takes to differ by lane is looped over lane by lane, a load at a time.
__device__ inline bool group_find(const int32_t* __restrict__ offsets, int E, int T, int BT, int tile, GroupTile& g) {
  const int lane = threadIdx.x & 63;
  int before = 0, e = -1, t0 = 0, t1 = 0;
  for (int e0 = 0; e0 < E && e < 0; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < E) group_range(offsets, e0 + lane, T, lo, hi);
    const int tiles = (hi - lo + BT - 1) / BT;
    int sum = tiles;   // inclusive prefix
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(sum, o, 64);
      if (lane >= o) sum = tile_sum(sum, up);
    }
    const uint64_t past = __ballot(before + sum > tile);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int start = before + (at > 0 ? __builtin_amdgcn_readlane(sum, at - 1) : 0);
      e = e0 + at;
      t0 = __builtin_amdgcn_readlane(lo, at) + (tile - start) * BT;
      t1 = __builtin_amdgcn_readlane(hi, at);
    }
    before = tile_sum(before, __builtin_amdgcn_readlane(sum, 63));
  }
  g.e = __builtin_amdgcn_readfirstlane(e);
  g.t0 = __builtin_amdgcn_readfirstlane(t0);
  g.t1 = __builtin_amdgcn_readfirstlane(t1);
  return g.e >= 0;
}

// How many tiles there are, by the whole wave.
__device__ inline int group_count(const int32_t* __restrict__ offsets, int E, int T, int BT) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int e = lane; e < E; e += 64) {
    int lo, hi;
    group_range(offsets, e, T, lo, hi);
    sum = tile_sum(sum, (hi - lo + BT - 1) / BT);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum = tile_sum(sum, __shfl_xor(sum, o, 64));
  return __builtin_amdgcn_readfirstlane(sum);
}

// The tiles as a table in a workspace: its size, and the launch that fills it
// (nm_group.hip).  Entry 0 holds the count, entries 1 .. count the tiles (e, t0,
// t1, 0); at most max_tiles of them.
inline size_t group_table_bytes(int64_t max_tiles) { return size_t(max_tiles + 1) * 16; }
hipError_t launch_group_tiles(const int32_t* offsets, int64_t E, int64_t T, int BT, int64_t max_tiles, int4* table,
                              hipStream_t s);

// Kernels of one tile a workgroup look for it themselves where the experts are few
// (under a microsecond for 64, behind the other workgroups' work; the table is a
// launch of 4 us before them), and read the table where they are many.
constexpr int64_t kFindExperts = 256;
struct GroupRows {
  const int32_t* offsets;   // null: one weight for all rows
  const int4* table;        // null: look for the tile
  int E;
  __device__ bool tile(int tt, int T, int BT, GroupTile& g) const {
    if (!offsets) {
      g = GroupTile{0, tt * BT, T};
      return true;
    }
    if (!table) return group_find(offsets, E, T, BT, tt, g);
    if (tt >= table[0].x) return false;
    const int4 e = table[1 + tt];
    g = GroupTile{e.x, e.y, e.z};
    return true;
  }
};

// The rows of a launch of tiles of BT tokens, its table (if any) filled in `workspace`
// of group_rows_bytes.
inline size_t group_rows_bytes(int64_t E, int64_t max_tiles) {
  return E > kFindExperts ? group_table_bytes(max_tiles) : 0;
}
inline hipError_t group_rows(const int32_t* offsets, int64_t E, int64_t T, int BT, int64_t max_tiles, void* workspace,
                             hipStream_t s, GroupRows& rows) {
  rows = GroupRows{offsets, nullptr, int(E)};
  if (!offsets || E <= kFindExperts) return hipSuccess;
  rows.table = static_cast<int4*>(workspace);
  return launch_group_tiles(offsets, E, T, BT, max_tiles, static_cast<int4*>(workspace), s);
}

}  // namespace nm
