// Prints the tiles that sgemm_orthogonalize takes for S, S S and a Z + P Z, a line for each three
// arguments: batch, rows and columns of Z.
#include <cstdio>
#include <cstdlib>

#include "orthogonalize.hpp"

int main(int argc, char **argv) {
  const char *const names[] = {"64x64", "128x128", "128x256"};
  for (int i = 1; i + 2 < argc; i += 3) {
    const int batch = atoi(argv[i]), m = atoi(argv[i + 1]), n = atoi(argv[i + 2]);
    auto name = [&](int a, int b, int k, bool symmetric) {
      return names[(int)sgemm::ortho_tile(a, b, k, symmetric, batch, 256)];
    };
    std::printf("%s %s %s\n", name(m, m, n, true), name(m, m, m, true), name(m, n, m, false));
  }
}
