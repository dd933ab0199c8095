// Host check of csrc/grouped_map.hpp: the division by up to 8 against exact
// division, and that the tiles of a group (tile_in_group over every position)
// are each reached once.
#include <cstdio>
#include <algorithm>
#include <random>
#include <vector>

#include "grouped_map.hpp"

int main() {
  long failures = 0;
  for (int d = 1; d <= 8; ++d) {
    for (int n = 0; n < (1 << 20); ++n) failures += sgemm::div_up_to_8(n, d) != n / d;
    for (int n = 1 << 20; n < (1 << 29) - 997; n += 997)
      failures += sgemm::div_up_to_8(n, d) != n / d;
    for (int n = (1 << 29) - 4096; n < (1 << 29); ++n)
      failures += sgemm::div_up_to_8(n, d) != n / d;
  }
  std::mt19937 rng(5);
  for (int c = 0; c < 4000; ++c) {
    const int tiles_m = 1 + (int)(rng() % 40), tiles_n = 1 + (int)(rng() % (c % 7 ? 50 : 1000));
    const sgemm::GroupMap map = sgemm::make_group_map(tiles_n);
    std::vector<int> seen(tiles_m * tiles_n);
    for (int in = 0; in < tiles_m * tiles_n; ++in) {
      int tm = -1, tn = -1;
      if (!sgemm::tile_in_group(map, in, tiles_m, tm, tn) || tm < 0 || tn < 0)
        ++failures;
      else
        ++seen[tm * tiles_n + tn];
    }
    for (int n : seen) failures += n != 1;
    // positions past the last tile are refused or inside the group
    for (int i = 0; i < 20; ++i) {
      int tm = 0, tn = 0;
      const int in = tiles_m * tiles_n + (int)(rng() % (1 << 28));
      if (sgemm::tile_in_group(map, in, tiles_m, tm, tn))
        failures += tm < 0 || tm >= tiles_m || tn < 0 || tn >= tiles_n;
    }
  }
  // the launched tile rows cover any way to divide M rows
  for (int c = 0; c < 20000; ++c) {
    const long M = 1 + rng() % 500, groups = 1 + rng() % 60, bm = 16L << rng() % 5;
    std::vector<long> cut(groups + 1);
    for (long &v : cut) v = rng() % (M + 1);
    long tiles = 0;
    std::sort(cut.begin(), cut.end());
    for (long g = 0; g < groups; ++g) tiles += (cut[g + 1] - cut[g] + bm - 1) / bm;
    failures += tiles > sgemm::group_tile_rows(M, groups, bm);
  }
  std::printf("failures %ld\n", failures);
  return failures != 0;
}
