// grouped_map.hpp -- work-group -> (group, tile) for products whose rows fall
// into groups of lengths that only the device knows.
//
// The host launches as many work-groups as any group lengths can need:
// sum_g ceil(rows_g / BM) <= M / BM + min(groups, M) rows of tiles.  Each
// wave reads the offsets itself (64 groups at a time, one per lane), sums the
// tile rows before each group with a wave-wide scan, and finds its tile;
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

// Group g's rows, clamped so that they lie in [0, M] whatever the offsets are.
__device__ __forceinline__ void group_range(const int64_t *offsets, int g, long M, long &first,
                                            long &last) {
  const long s = offsets[g], e = offsets[g + 1];
  first = s < 0 ? 0 : (s > M ? M : s);
  last = e < first ? first : (e > M ? M : e);
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The tile of work-group blockIdx.x: tiles of bm rows, tiles_n of them across,
// group after group; inside a group a raster of group_m tile rows walked
// column by column (TileMap's order).  All lanes of all waves get the same
// answer.
__device__ __forceinline__ GroupTile group_tile(const int64_t *offsets, int groups, long M, int bm,
                                                int tiles_n, int group_m) {
  const int lane = threadIdx.x % kWave;
  auto tiles_of = [&](int g, long &first, long &last) {
    first = last = 0;
    if (g < groups) group_range(offsets, g, M, first, last);
    return (int)((last - first + bm - 1) / bm);
  };
  long first, last;
  int scan = wave_scan(tiles_of(lane, first, last), lane);  // the first 64 groups
  int total = __builtin_amdgcn_readlane(scan, kWave - 1);
  for (int b = kWave; b < groups; b += kWave) {
    long f, l;
    const int s = wave_scan(tiles_of(b + lane, f, l), lane);
    total += __builtin_amdgcn_readlane(s, kWave - 1);
  }
  GroupTile t;
  t.valid = false;
  t.g = t.rows = t.tm = t.tn = 0;
  t.row0 = 0;
  const unsigned tiles = (unsigned)total * (unsigned)tiles_n;
  if (total <= 0 || blockIdx.x >= tiles) return t;
  const unsigned pos = (unsigned)xcd_contiguous_id(blockIdx.x, tiles);
  const int q = (int)(pos / (unsigned)tiles_n);  // rows of tiles before this one's row start
  int base = 0;                                  // tile rows of earlier blocks of 64 groups
  int block = 0;
  for (;; block += kWave) {
    const int end = base + __builtin_amdgcn_readlane(scan, kWave - 1);
    if (q < end || block + kWave >= groups) break;
    base = end;
    scan = wave_scan(tiles_of(block + kWave + lane, first, last), lane);
  }
  const unsigned long long after = __ballot(base + scan > q);
  if (after == 0) return t;  // offsets that decrease can leave no group for it
  const int l = __builtin_ctzll(after);
  t.g = block + l;
  group_range(offsets, t.g, M, first, last);
  t.row0 = first;
  t.rows = (int)(last - first);
  const int tiles_m = (t.rows + bm - 1) / bm;
  const int before = l == 0 ? base : base + __builtin_amdgcn_readlane(scan, l > 0 ? l - 1 : 0);
  const unsigned in = pos - (unsigned)before * (unsigned)tiles_n;
  const unsigned per = (unsigned)group_m * (unsigned)tiles_n;
  const int first_row = (int)(in / per) * group_m;
  const unsigned r = in % per;
  const int high = min(group_m, tiles_m - first_row);
  if (first_row < 0 || high <= 0) return t;
  t.tn = (int)(r / (unsigned)high);
  t.tm = first_row + (int)(r % (unsigned)high);
  t.valid = t.tn < tiles_n && t.tm < tiles_m;
  return t;
}

// The group with `rank` longer ones before it (equal ones in their order),
// among up to 64 groups; with more groups, group `rank`.
__device__ __forceinline__ int group_by_length(const int64_t *offsets, int groups, long M,
                                               int rank) {
  if (groups > kWave) return rank;
  const int lane = threadIdx.x % kWave;
  long first = 0, last = -1;
  if (lane < groups) group_range(offsets, lane, M, first, last);
  const int mine = (int)(last - first);  // -1 past the last group
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
