// Host check of csrc/grouped_map.hpp's clamp of a group's rows: whatever the
// offsets are, they lie in [0, M] in order, and offsets that need no clamp are
// taken as they are.
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>

#include "grouped_map.hpp"

int main() {
  long failures = 0;
  std::mt19937_64 rng(8);
  const int64_t lowest = std::numeric_limits<int64_t>::min(),
                highest = std::numeric_limits<int64_t>::max();
  for (int c = 0; c < 200000; ++c) {
    const int M = c % 3 == 0 ? std::numeric_limits<int>::max() : (int)(rng() % 50);
    int64_t at[9];
    for (int64_t &v : at) {
      const int64_t near = (int64_t)(rng() % 120) - 60;
      const int64_t some[] = {lowest, highest, -1, 0, M, M + 1LL, near, (int64_t)rng(),
                              (int64_t)(rng() % (M + 1LL))};
      v = some[rng() % 9];
    }
    for (int g = 0; g < 8; ++g) {
      int first = -7, last = -7;
      sgemm::group_range(at, g, M, first, last);
      failures += !(0 <= first && first <= last && last <= M);
      const int64_t s = at[g], e = at[g + 1];
      if (0 <= s && s <= e && e <= M) failures += first != s || last != e;
      if (s >= M || e <= s) failures += first != last;
      if (0 <= s && s <= M && e > M) failures += first != s || last != M;
    }
  }
  std::printf("failures %ld\n", failures);
  return failures != 0;
}
