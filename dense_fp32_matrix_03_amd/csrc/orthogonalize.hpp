// orthogonalize.hpp -- matrices held as two half-precision pieces, and the
// launchers of the Newton-Schulz steps on them (include/sgemm_orthogonalize.h).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.hpp"

namespace sgemm {

// A batch of matrices in pieces: [cols / 32][rows] blocks of 128 bytes, 32 high
// pieces of a row and then 32 low ones, the last columns padded with zeros.  A
// value is (high + low) 2^(e - kHeldTop) with the row's e (RowScale).
struct SplitMatrix {
  char *at;
  int rows, cols;
  long stride;  // bytes from one matrix to the next
  // Where the high piece of (r, c) lies; the low one is 64 bytes after it.
  __device__ __forceinline__ char *place(int batch, int r, int c) const {
    return at + batch * stride + ((long)(c / 32) * rows + r) * 128 + c % 32 * 2;
  }
  __host__ __device__ __forceinline__ int padded() const { return (cols + 31) / 32 * 32; }
};
inline long split_bytes(long rows, long cols) { return (cols + 31) / 32 * rows * 128; }

// The range of a row of a held matrix: no element reaches 2^e.  A row of one size among
// rows of another keeps its digits only if e goes by the row.  e is known before the row
// is: a product with Z's row or from the left can make no more of its norm than the
// polynomials' bounds allow, so that every e is a constant of the step past the exponent
// of the norm that Z's row had when it was last looked at, and at most a constant of
// the step, as the whole matrix has it.
constexpr int kHeldTop = 15;  // a held element is below 2^15, half of half precision's range
constexpr int kLeastExponent = -100;
struct RowScale {
  const signed char *norm;  // [batch][count]: the norm of rows i with this i >> shift is below 2^norm
  int count, shift;
  int add, cap;
  __device__ __forceinline__ unsigned index(int batch, int row) const {  // below 2^29
    return (unsigned)batch * (unsigned)count + (unsigned)(row >> shift);
  }
  __device__ __forceinline__ int exponent(int norm) const {
    return max(min(norm + add, cap), kLeastExponent);
  }
};
// A norm's exponent, from the bits of the largest magnitude of a row and the exponent of
// the root of its length.
__host__ __device__ __forceinline__ signed char norm_exponent(unsigned top, int length) {
  const int e = (int)(top >> 23) - 126 + length;
  return (signed char)(e < -127 ? -127 : e > 127 ? 127 : e);
}

// The sum of squares, in parts, of every matrix of the batch.
struct OrthoNormArgs {
  int M, N;
  const void *X;
  long ldx, strideX;
  double *parts;  // [batch][n_parts]
  int n_parts;
};
constexpr int kNormRun = 512;    // elements of a row that a wave adds up at a time
constexpr int kNormParts = 256;  // parts, at most: a work-group each, of 16 such runs or more
hipError_t launch_ortho_norm(const OrthoNormArgs &p, bool bf16, int batch, hipStream_t s);

// 1 / (|X| + eps) of every matrix, and the norms' exponents of the rows and columns of X
// times that.
struct OrthoSizesArgs {
  int M, N;
  const void *X;
  long ldx, strideX;
  float eps;
  // A work-group has `band` rows by 512 columns, and writes its sum of squares and the
  // largest magnitudes of its rows and columns.
  int band, bands, runs;
  double *parts;                    // [batch][bands][runs]
  unsigned *row_parts, *col_parts;  // [batch][runs][M], [batch][bands][N]
  bool summed;                      // by a launch of its own: very many parts
  double *scale;                    // [batch], where summed; null: 1
  signed char *rows, *cols;         // as in RowScale
  int row_shift, col_shift;         // both 0 but where summed
  int row_length, col_length;       // exponents of the roots of N and M
};
inline int sizes_runs(long N) { return (int)((N + kNormRun - 1) / kNormRun); }
// A multiple of 16, for about 224 work-groups: with what rounding adds, 65535 matrices
// stay below 2^32 work-items.
inline int sizes_band(long M, long N) {
  const long share = (M * sizes_runs(N) + 223) / 224;
  return (int)((share < M ? share : M) + 15) / 16 * 16;
}
inline int sizes_bands(long M, long N) { return (int)((M + sizes_band(M, N) - 1) / sizes_band(M, N)); }
constexpr int kMostSizeParts = 24;  // of a row and of a column that each block adds up for itself
hipError_t launch_ortho_sizes(const OrthoSizesArgs &p, bool bf16, int batch, hipStream_t s);

// X times its scale, in pieces, as it is and transposed.
struct OrthoSplitArgs {
  OrthoSizesArgs x;
  RowScale row_scale, col_scale;  // of X's rows and columns
  SplitMatrix rows, cols;         // M x N and N x M
};
hipError_t launch_ortho_split(const OrthoSplitArgs &p, bool bf16, int batch, hipStream_t s);

// The norms' exponents of the rows and columns of z, which is held by z_scale.  p: M and N of
// z, rows, cols and what they go by; row_parts and col_parts, one after the other, are room.
hipError_t launch_ortho_look(const OrthoSizesArgs &p, const SplitMatrix &z, const RowScale &z_scale,
                             int batch, hipStream_t s);

// D = f1 A B^T + f2 E, of A's rows by B's rows.  E is held twice, by its rows and, transposed,
// by its columns, as B is: an element is taken from the copy whose range is the smaller.
struct OrthoProductArgs {
  SplitMatrix a, b;
  RowScale a_scale, b_scale;
  SplitMatrix e, e_t;  // e.at == null: none.  e may be d
  RowScale e_scale;    // valid in any case, as the two below
  float f1, f2;
  SplitMatrix d, d_t;  // D as it is and transposed; at == null: not written
  RowScale d_scale, d_t_scale;
  // The last product's D times alpha instead, in a user's type: element (m, n) at m ld +
  // n, or at n ld + m.
  void *Y;
  long ldy, strideY;
  bool y_transposed;
  float alpha;
  // What the launch moves besides, 16 bytes at a time.
  const char *move_from;
  char *move_to;
  unsigned moves;
};
// symmetric: D is symmetric, A and B the same, and one half of D is computed.
hipError_t launch_ortho_product(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                                int cus, hipStream_t s);

// The tile by times in microseconds, n the tiles for each of the chip's compute units,
// nk slices.  Measured on 256 compute units (S = Z Z^T, or a Z + P Z; m x n of Z, tiles
// of 64 x 64 / 128 x 128 / 128 x 256):
//   S    1024 x 1024      10.0 / 18.8       2048 x 2048      45 / 41
//        2600 x 2600      91 / 58           2048 x 4096      80 / 58
//        16 of 512 x 512  17.5 / 16.1       1500 x 1500      22 / 26
//   a Z + P Z
//        1024 x 1024      13.3 / 22 / 34    2048 x 2048      64 / 54 / 69
//        2600 x 2600      132 / 116 / 107   2048 x 4096      122 / 103 / 92
//        16 of 512 x 512  28 / 24 / 29      1500 x 1500      36 / 32 / 47
// A tile of 64 x 64 is bound by what the caches deliver, 85 bytes a nanosecond and
// compute unit; larger ones by the matrix cores, at the power limit once the chip is
// full (1.1 PFLOP/s of half precision, where a large library product has 1.3).
enum class OrthoTile { k64, k128, k128x256 };
inline OrthoTile ortho_tile(int rows_a, int rows_b, int cols, bool symmetric, int batch, int cus) {
  const double nk = (cols + 31) / 32;
  auto tiles = [&](int bm, int bn) {
    const double tm = (rows_a + bm - 1) / bm, tn = (rows_b + bn - 1) / bn;
    return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn) / cus;
  };
  const double n64 = tiles(64, 64), n128 = tiles(128, 128);
  const double c64 = ceil(n64) * (0.2 * nk + 2);
  if (symmetric) {
    const double c128 = ceil(n128) * (0.38 * nk + 6 + 12 * fmin(n128, 1));
    return c64 <= c128 ? OrthoTile::k64 : OrthoTile::k128;
  }
  const double c128 =
      fmax(1, (ceil(n128) + n128) / 2) * ((0.38 + 0.22 * fmin(n128, 1)) * nk + 11);
  const double n256 = tiles(128, 256);
  const double c256 = ceil(n256) * (0.85 * nk + 12 + 50 * fmin(fmax(n256 - 0.6, 0), 0.4));
  if (c64 <= c128 && c64 <= c256) return OrthoTile::k64;
  return c128 <= c256 ? OrthoTile::k128 : OrthoTile::k128x256;
}

// Matrices of at most kShort rows (Z, m x n): a launch for Z and S's parts, then one for
// each step (orthogonalize_short.hip).  A slab is `blocks` times 64 columns.
constexpr int kShort = 64;
// At most 16 slabs, since each work-group adds up all their parts, 32 where a work-group
// would have many blocks one after the other.  16 / 32 slabs: 32 of 64 x 4096 225 / 315 us,
// 1 of 32 x 4096 116 / 100, 64 x 100000 1800 / 951.  The batch would tell the first two
// apart, but the slabs are the order in which S is summed, and a matrix has the same bits
// whatever the batch around it: what a batch loses by 32 is more than one gains.
inline int short_blocks(int n) {
  const int slabs = n <= 8192 ? 16 : 32;
  return ((n + 63) / 64 + slabs - 1) / slabs;
}
inline int short_slabs(int n) { return ((n + 63) / 64 + short_blocks(n) - 1) / short_blocks(n); }
struct OrthoShortArgs {
  int m, n, slabs, blocks;
  FastDiv by_m;
  // Z(r, c) of X at r xr + c xc, of Y at r yr + c yc; one of the two is 1.
  const void *X;
  long xr, xc, strideX;
  void *Y;
  long yr, yc, strideY;
  OrthoNormArgs norm;
  float eps, a, b, c, alpha;
  const float *z_in, *part_in;  // [batch][m][n]; [batch][slabs][m][m]
  float *z_out, *part_out;
};
hipError_t launch_ortho_short(const OrthoShortArgs &p, bool first, bool last, bool bf16, int batch,
                              hipStream_t s);

}  // namespace sgemm
