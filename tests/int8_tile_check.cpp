// Prints the kernel that an 8-bit product of a held A takes, a line for each four arguments:
// groups (0: not grouped), M, N, K.
#include <cstdio>
#include <cstdlib>

#include "int8.hpp"

int main(int argc, char **argv) {
  const char *const names[] = {"64/2", "64/3", "64/4", "128", "128x256", "256"};
  static const int64_t some = 0;
  for (int i = 1; i + 3 < argc; i += 4) {
    sgemm::Int8Args p{};
    const int groups = atoi(argv[i]);
    p.groups = groups ? groups : 1;
    p.M = atoi(argv[i + 1]);
    p.N = atoi(argv[i + 2]);
    p.K = atoi(argv[i + 3]);
    p.offsets = groups ? &some : nullptr;
    std::printf("%s\n", sgemm::int8_few_rows(p, 256) ? "rows" : names[(int)sgemm::int8_tile(p, 256)]);
  }
}
