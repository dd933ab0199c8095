// grouped_map.hpp -- work-group -> (group, tile) for products whose rows fall
// into groups of lengths that only the device knows.
//
// The host launches as many work-groups as any group lengths can need:
// sum_g ceil(rows_g / BM) <= M / BM + min(groups, M) rows of tiles.  Each
// wave reads the offsets itself (up to 64 groups: one per lane), sums the tile
// rows before each group with a wave-wide scan, and finds its tile;
// work-groups past the last tile leave.  That costs about one memory round
// trip, against a launch of its own (and memory between the two) for a kernel
// that would write the map out.  The total has to be known before the tile,
// because the renumbering that gives each XCD a contiguous range of tiles
// must cover the tiles there are: over the launched range the last XCDs would
// get little but idle work-groups.
#pragma once

#include "common.hpp"

namespace sgemm {

struct GroupTile {
  bool valid;
  int g;         // group
  long row0;     // first row of the group
  int rows;      // rows of the group
  int tm, tn;    // tile inside the group
};

// Group g's rows, clamped so that they lie in [0, M] whatever the offsets are
// (M < 2^31).
__device__ __forceinline__ void group_range(const int64_t *offsets, int g, int M, int &first,
                                            int &last) {
  const int64_t s = offsets[g], e = offsets[g + 1];
  first = s < 0 ? 0 : (s > M ? M : (int)s);
  last = e < first ? first : (e > M ? M : (int)e);
}

// Inclusive sum over the lanes up to this one, by moves inside rows of 16 lanes
// and from row to row (no LDS: each step is one instruction, where a shuffle
// waits for LDS six times over).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1 lane before, in a row
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // rows 1, 3: the row before's last
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // rows 2, 3: lane 31
  return v;
}

// The tile of work-group blockIdx.x: tiles of bm rows, tiles_n of them across,
// group after group; inside a group a raster of group_m tile rows walked
// column by column (TileMap's order).  All lanes of all waves get the same
// answer.  Lane l sums `per` consecutive groups; where that is more than one,
// the lane's groups are then told apart by a second sum over lanes.
__device__ __forceinline__ GroupTile group_tile(const int64_t *offsets, int groups, int M, int bm,
                                                int tiles_n, int group_m) {
  const int lane = threadIdx.x % kWave;
  const int per = (groups + kWave - 1) / kWave;
  auto tiles_of = [&](int g, int &first, int &last) {
    first = last = 0;
    if (g < groups) group_range(offsets, g, M, first, last);
    return (last - first + bm - 1) / bm;
  };
  GroupTile t;
  t.valid = false;
  t.g = t.rows = t.tm = t.tn = 0;
  t.row0 = 0;
  int first, last, tiles = tiles_of(lane * per, first, last);
  for (int i = 1; i < per; ++i) {
    int f, l;
    tiles += tiles_of(lane * per + i, f, l);
  }
  int scan = wave_scan(tiles);
  const int total = __builtin_amdgcn_readlane(scan, kWave - 1);
  const unsigned all = (unsigned)total * (unsigned)tiles_n;
  if (total <= 0 || blockIdx.x >= all) return t;
  const unsigned pos = (unsigned)xcd_contiguous_id(blockIdx.x, all);
  const int q = (int)(pos / (unsigned)tiles_n);  // tile rows before this tile's row start
  // Offsets that decrease can make these sums meaningless: whatever group and
  // tile come out are checked against the group's own range at the end.
  unsigned long long after = __ballot(scan > q);
  if (after == 0) return t;
  int l = __builtin_ctzll(after);
  int before = l > 0 ? __builtin_amdgcn_readlane(scan, l > 0 ? l - 1 : 0) : 0;
  t.g = l;
  if (per > 1) {
    const int g0 = l * per;
    tiles = lane < per ? tiles_of(g0 + lane, first, last) : 0;
    scan = wave_scan(tiles) + before;
    after = __ballot(scan > q);
    if (after == 0) return t;
    l = __builtin_ctzll(after);
    before = l > 0 ? __builtin_amdgcn_readlane(scan, l > 0 ? l - 1 : 0) : before;
    t.g = g0 + l;
  }
  if (t.g >= groups) return t;
  t.row0 = __builtin_amdgcn_readlane(first, l);
  t.rows = __builtin_amdgcn_readlane(last, l) - (int)t.row0;
  const int tiles_m = (t.rows + bm - 1) / bm;
  const unsigned in = pos - (unsigned)before * (unsigned)tiles_n;
  const unsigned per_raster = (unsigned)group_m * (unsigned)tiles_n;
  const int first_row = (int)(in / per_raster) * group_m;
  const unsigned r = in % per_raster;
  const int high = min(group_m, tiles_m - first_row);
  if (first_row < 0 || high <= 0) return t;
  t.tn = (int)(r / (unsigned)high);
  t.tm = first_row + (int)(r % (unsigned)high);
  t.valid = t.tn < tiles_n && t.tm < tiles_m;
  return t;
}

// The group with `rank` longer ones before it (equal ones in their order),
// among up to 64 groups; with more groups, group `rank`.
__device__ __forceinline__ int group_by_length(const int64_t *offsets, int groups, int M,
                                               int rank) {
  if (groups > kWave) return rank;
  const int lane = threadIdx.x % kWave;
  int first = 0, last = -1;
  if (lane < groups) group_range(offsets, lane, M, first, last);
  const int mine = last - first;  // -1 past the last group
  int before = 0;
  for (int g = 0; g < groups; ++g) {
    const int other = __builtin_amdgcn_readlane(mine, g);
    before += other > mine || (other == mine && g < lane);
  }
  return __builtin_ctzll(__ballot(before == rank && lane < groups));
}

// Tile rows that a launch must provide for M rows in `groups` groups.
inline long group_tile_rows(long M, long groups, long bm) {
  return M / bm + (groups < M ? groups : M);
}

}  // namespace sgemm
