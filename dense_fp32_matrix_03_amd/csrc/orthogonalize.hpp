// orthogonalize.hpp -- matrices held as two half-precision pieces, and the
// launchers of the Newton-Schulz steps on them (include/sgemm_orthogonalize.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace sgemm {

// A batch of matrices in pieces: [cols / 32][rows] blocks of 128 bytes, 32 high
// pieces of a row and then 32 low ones, the last columns padded with zeros.  A
// value is (high + low) 2^-s with an s that the host keeps.
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

// X 2^shift / (|X| + eps), in pieces, as it is and transposed.
struct OrthoSplitArgs {
  OrthoNormArgs x;
  float eps;
  int shift;
  SplitMatrix rows, cols;  // M x N and N x M
};
hipError_t launch_ortho_split(const OrthoSplitArgs &p, bool bf16, int batch, hipStream_t s);

// D = f1 A B^T + f2 E, of A's rows by B's rows.
struct OrthoProductArgs {
  SplitMatrix a, b;
  SplitMatrix e_t;  // E transposed; at == null: none
  float f1, f2;
  SplitMatrix d, d_t;  // D as it is and transposed; at == null: not written
  // The last product's D instead, in a user's type: element (m, n) at m ld + n, or
  // at n ld + m.
  void *Y;
  long ldy, strideY;
  bool y_transposed;
};
// symmetric: D is symmetric, A and B the same, and one half of its tiles is
// computed.
hipError_t launch_ortho_product(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                                int cus, hipStream_t s);

// Matrices of at most kShort rows (Z, m x n): a launch for Z and S's parts, then one for
// each step (orthogonalize_short.hip).  A slab is `blocks` times 64 columns.
constexpr int kShort = 64;
// At most 16 slabs, since each work-group adds up all their parts, 32 where a work-group
// would have many blocks one after the other.  16 / 32 slabs: 32 of 64 x 4096 225 / 315 us,
// 1 of 32 x 4096 116 / 100, 64 x 100000 1800 / 951.
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
