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

constexpr int kGroupRaster = 8;  // tile rows of a raster strip inside a group

// What the host knows of the map: tiles across, and divisors by them, so that a
// work-group's prologue multiplies by constants instead of dividing.
struct GroupMap {
  int tiles_n;
  FastDiv by_tiles_n, by_strip;  // strip: kGroupRaster tiles_n tiles
};

inline GroupMap make_group_map(int tiles_n) {  // host side
  return GroupMap{tiles_n, make_fast_div(tiles_n), make_fast_div(kGroupRaster * tiles_n)};
}

// n / d for 1 <= d <= 8 and n < 2^29: with m = ceil(2^32 / d), m d exceeds 2^32
// by less than d, so floor(n m / 2^32) is exact while n (m d - 2^32) < 2^32.
__host__ __device__ __forceinline__ int div_up_to_8(int n, int d) {
  const unsigned m = d == 2   ? 0x80000000u
                     : d == 3 ? 0x55555556u
                     : d == 4 ? 0x40000000u
                     : d == 5 ? 0x33333334u
                     : d == 6 ? 0x2aaaaaabu
                     : d == 7 ? 0x24924925u
                              : 0x20000000u;
  return d == 1 ? n : (int)((unsigned long long)(unsigned)n * m >> 32);
}

// Tile `in` of a group with tiles_m rows of tiles: strips of kGroupRaster tile
// rows walked column by column (TileMap's order).  False if it has no such
// tile.
__host__ __device__ __forceinline__ bool tile_in_group(const GroupMap &map, int in, int tiles_m,
                                                       int &tm, int &tn) {
  const int strip = map.by_strip(in), r = in - strip * (kGroupRaster * map.tiles_n);
  const int left = tiles_m - strip * kGroupRaster;
  const int high = left < kGroupRaster ? left : kGroupRaster;
  if (high <= 0) return false;
  tn = div_up_to_8(r, high);
  tm = strip * kGroupRaster + (r - tn * high);
  return tn < map.tiles_n && tm < tiles_m;
}

struct GroupTile {
  bool valid;
  int g;         // group
  long row0;     // first row of the group
  int rows;      // rows of the group
  int tm, tn;    // tile inside the group
};

// Group g's rows, clamped so that they lie in [0, M] whatever the offsets are
// (M < 2^31).
__host__ __device__ __forceinline__ void group_range(const int64_t *offsets, int g, int M,
                                                     int &first, int &last) {
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

// The tile of work-group blockIdx.x: tiles of bm rows (a power of two), tiles_n
// of them across, group after group, in tile_in_group's order.  All lanes of all waves get the same
// answer.  Lane l sums `per` consecutive groups; where that is more than one,
// the lane's groups are then told apart by a second sum over lanes.
__device__ __forceinline__ GroupTile group_tile(const int64_t *offsets, int groups, int M, int bm,
                                                const GroupMap &map) {
  const int tiles_n = map.tiles_n;
  const int lane = threadIdx.x % kWave;
  const int per = (groups + kWave - 1) / kWave;
  auto tiles_of = [&](int g, int &first, int &last) {
    first = last = 0;
    if (g < groups) group_range(offsets, g, M, first, last);
    return (last - first + bm - 1) / bm;  // bm is a constant power of two
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
  if (pos >= 1u << 29) return t;       // no launch has as many; keeps the divisions in range
  const int q = map.by_tiles_n((int)pos);  // tile rows before this tile's row start
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
  const int in = (int)(pos - (unsigned)before * (unsigned)tiles_n);
  if (in < 0 || in >= 1 << 29) return t;
  t.valid = tile_in_group(map, in, tiles_m, t.tm, t.tn);
  return t;
}

// The group with `rank` longer ones before it (equal ones in their order),
// among up to 64 groups; with more groups, group `rank`.  And its rows.
__device__ __forceinline__ int group_by_length(const int64_t *offsets, int groups, int M, int rank,
                                               int &first, int &last) {
  if (groups > kWave) {
    group_range(offsets, rank, M, first, last);
    return rank;
  }
  const int lane = threadIdx.x % kWave;
  int f = 0, l = 0;
  if (lane < groups) group_range(offsets, lane, M, f, l);
  // Bit by bit from the highest: the lanes of `same` agree with the group sought
  // in the bits seen so far.
  unsigned long long same = __ballot(lane < groups);
  for (int bit = 31 - __builtin_clz(M | 1); bit >= 0; --bit) {
    const unsigned long long ones = same & __ballot(((l - f) >> bit & 1) != 0);
    const int longer = __builtin_popcountll(ones);
    same = rank < longer ? ones : same & ~ones;
    rank = rank < longer ? rank : rank - longer;
  }
  const int at = __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32),
                                           __builtin_amdgcn_mbcnt_lo((unsigned)same, 0));
  const int g = __builtin_ctzll(same & __ballot(at == rank));
  first = __builtin_amdgcn_readlane(f, g);
  last = __builtin_amdgcn_readlane(l, g);
  return g;
}

// Tile rows that a launch must provide for M rows in `groups` groups.
inline long group_tile_rows(long M, long groups, long bm) {
  return M / bm + (groups < M ? groups : M);
}

}  // namespace sgemm
