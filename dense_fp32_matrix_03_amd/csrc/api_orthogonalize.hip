// api_orthogonalize.hip -- the C interface declared in
// include/sgemm_orthogonalize.h: argument checks, the workspace's layout, the
// ranges of the steps' matrices and the launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_internal.hpp"
#include "orthogonalize.hpp"
#include "sgemm_orthogonalize.h"

namespace {

using sgemm_api::kMaxDim;
using sgemm_api::kMaxWorkItems;

constexpr int64_t kMaxSize = int64_t(1) << 20;  // of a matrix: a slice of it is below 2^31 bytes
constexpr int64_t kMaxBatch = 65535;            // the second dimension of a launch
constexpr int64_t kMaxSteps = 64;
// Steps after which the rows and columns of Z are looked at again: until then they may
// have grown by the polynomials' bound, 3.44 a step for common ones, where those that
// are parallel to large ones did not.  8 such steps are 2^14.3 of the 2^17 that a held
// element may lie below its row's bound with all of its digits.
constexpr int64_t kLookAgain = 8;
constexpr int64_t kLooks = (kMaxSteps - 1) / kLookAgain;

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool bad_type(int type) { return type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16; }
unsigned size_of(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// The workspace: Z and Z transposed twice (a step reads one and writes the other), S and P
// in pieces, Z transposed and S in floats; sizes of rows and columns, in parts, and then once for
// each look at them.  Short matrices: the parts of the norms, and Z and the parts of S
// twice.
struct Layout {
  int m, n;
  int64_t z, zt, s;     // bytes of a matrix
  int64_t parts;        // of a norm
  int64_t row_parts, col_parts, rows, cols;  // bytes of a matrix
  int64_t total;
  // Where m is short: Z and S's parts, twice each.
  bool is_short;
  int64_t short_z, short_parts;
  Layout(int64_t batch, int64_t M, int64_t N) {
    m = (int)(M < N ? M : N);
    n = (int)(M < N ? N : M);
    z = sgemm::split_bytes(m, n);
    zt = sgemm::split_bytes(n, m);
    s = sgemm::split_bytes(m, m);
    is_short = m <= sgemm::kShort;
    if (is_short) {
      parts = tiles(M * tiles(N, sgemm::kNormRun), 16);
      if (parts > sgemm::kNormParts) parts = sgemm::kNormParts;
    } else {
      parts = (int64_t)sgemm::sizes_bands(M, N) * sgemm::sizes_runs(N);
    }
    row_parts = 4 * sgemm::sizes_runs(N) * M;
    col_parts = 4 * sgemm::sizes_bands(M, N) * N;
    rows = 4 * (1 + kLooks) * M;
    cols = 4 * (1 + kLooks) * N;
    short_z = 4 * (int64_t)m * n;
    short_parts = 4 * (int64_t)m * m * sgemm::short_slabs(n);
    total = batch * (8 * parts + (is_short ? 2 * (short_z + short_parts)
                                           : 8 + z + 3 * zt + 3 * s + row_parts + col_parts + rows +
                                                 cols));
  }
};

int check_sizes(int64_t batch, int64_t M, int64_t N) {
  if (batch < 0 || M < 0 || N < 0) return SGEMM_ERR_INVALID_VALUE;
  if (M > kMaxSize || N > kMaxSize || batch > kMaxBatch) return SGEMM_ERR_TOO_LARGE;
  // Work-groups of 256 for tiles of 64 x 64, of either S or Z.
  const int64_t m = M < N ? M : N, n = M < N ? N : M;
  if (batch > 0 && tiles(m, 64) * tiles(n, 64) > (int64_t(1) << 23) / batch) return SGEMM_ERR_TOO_LARGE;
  return SGEMM_OK;
}

// The largest |a s + b s^3 + c s^5| for 0 <= s <= top: at the end, or where the
// derivative a + 3 b t + 5 c t^2 with t = s^2 is 0.
double largest(double a, double b, double c, double top) {
  auto at = [&](double s) { return fabs(s * (a + s * s * (b + s * s * c))); };
  double most = at(top);
  const double disc = 9 * b * b - 20 * a * c;
  double roots[3] = {0, 0, 0};
  if (disc >= 0) {
    // Both roots without cancellation: q / (5 c) and a / q.
    const double q = -0.5 * (3 * b + (b < 0 ? -1 : 1) * sqrt(disc));
    if (c != 0) roots[0] = q / (5 * c);
    if (q != 0) roots[1] = a / q;
  }
  if (b != 0) roots[2] = -a / (3 * b);  // c == 0 (for others any point is a fair one)
  for (double t : roots)
    if (t > 0 && t < top * top) most = fmax(most, at(sqrt(t)));
  return most;
}

// The largest |a + b t + c t^2| for 0 <= t <= top: how much a step can make of a vector.
double largest_growth(double a, double b, double c, double top) {
  auto at = [&](double t) { return fabs(a + t * (b + t * c)); };
  double most = fmax(at(0), at(top));
  const double t = c != 0 ? -b / (2 * c) : 0;
  return t > 0 && t < top ? fmax(most, at(t)) : most;
}

// The least e with bound < 2^e, with room for roundings.
int exponent_of(double bound) {
  if (!(bound > 0)) return -1000;
  int e;
  frexp(bound * 1.02, &e);
  return e;
}

// The launches for a short matrix.
int short_steps(const Layout &l, int64_t batch, int64_t M, int64_t N, int64_t steps, int64_t sets,
                const float *coefficients, float eps, float alpha, int typeX, const void *X,
                int64_t ldx, int64_t strideX, int typeY, void *Y, int64_t ldy, int64_t strideY,
                void *workspace, hipStream_t s) {
  const bool tall = M > N;
  char *at = static_cast<char *>(workspace);
  auto take = [&](int64_t bytes) {
    char *const from = at;
    at += batch * bytes;
    return reinterpret_cast<float *>(from);
  };
  sgemm::OrthoShortArgs p{};
  p.m = l.m;
  p.n = l.n;
  p.blocks = sgemm::short_blocks(l.n);
  p.slabs = sgemm::short_slabs(l.n);
  p.by_m = sgemm::make_fast_div(l.m);
  p.X = X;
  p.xr = tall ? 1 : ldx;
  p.xc = tall ? ldx : 1;
  p.strideX = strideX;
  p.Y = Y;
  p.yr = tall ? 1 : ldy;
  p.yc = tall ? ldy : 1;
  p.strideY = strideY;
  p.norm = {(int)M, (int)N, X, ldx, strideX, reinterpret_cast<double *>(take(8 * l.parts)),
            (int)l.parts};
  p.eps = eps;
  p.alpha = alpha;
  float *const z[2] = {take(l.short_z), take(l.short_z)};
  float *const part[2] = {take(l.short_parts), take(l.short_parts)};
  p.z_out = z[0];
  p.part_out = part[0];
  const bool x_bf16 = typeX == SGEMM_TYPE_BF16, y_bf16 = typeY == SGEMM_TYPE_BF16;
  hipError_t err = sgemm::launch_ortho_norm(p.norm, x_bf16, (int)batch, s);
  if (err == hipSuccess) err = sgemm::launch_ortho_short(p, true, false, x_bf16, (int)batch, s);
  for (int64_t k = 0; k < steps && err == hipSuccess; ++k) {
    const float *c = coefficients + (sets == 1 ? 0 : 3 * k);
    p.a = c[0];
    p.b = c[1];
    p.c = c[2];
    p.z_in = z[k % 2];
    p.part_in = part[k % 2];
    p.z_out = z[1 - k % 2];
    p.part_out = part[1 - k % 2];
    err = sgemm::launch_ortho_short(p, false, k + 1 == steps, y_bf16, (int)batch, s);
  }
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int64_t sgemm_orthogonalize_workspace_size(int64_t batch, int64_t M, int64_t N) {
  const int rc = check_sizes(batch, M, N);
  if (rc != SGEMM_OK) return rc;
  return batch == 0 || M == 0 || N == 0 ? 0 : Layout(batch, M, N).total;
}

int sgemm_orthogonalize(int64_t batch, int64_t M, int64_t N, int64_t steps, int64_t sets,
                        const float *coefficients, float eps, float alpha, int typeX,
                        const void *X, int64_t ldx, int64_t strideX, int typeY, void *Y,
                        int64_t ldy, int64_t strideY, void *workspace, int64_t workspace_bytes,
                        void *stream) {
  const int sizes = check_sizes(batch, M, N);
  if (sizes == SGEMM_ERR_INVALID_VALUE || bad_type(typeX) || bad_type(typeY) || steps < 1 ||
      steps > kMaxSteps || (sets != 1 && sets != steps) || !coefficients || !(eps >= 0.f) ||
      !isfinite(eps) || !isfinite(alpha))
    return SGEMM_ERR_INVALID_VALUE;
  if (ldx < (N > 1 ? N : 1) || ldy < (N > 1 ? N : 1) || strideX < 0 || strideY < 0)
    return SGEMM_ERR_INVALID_VALUE;
  if (batch > 1 && M > 0 && N > 0 && (__int128)(M - 1) * ldy + N > strideY)
    return SGEMM_ERR_INVALID_VALUE;
  // The largest singular value before each step and after the last.
  double bound[kMaxSteps + 1];
  bound[0] = 1.0;
  for (int64_t k = 0; k < steps; ++k) {
    const float *c = coefficients + (sets == 1 ? 0 : 3 * k);
    if (!isfinite(c[0]) || !isfinite(c[1]) || !isfinite(c[2])) return SGEMM_ERR_INVALID_VALUE;
    // Roundings move a singular value a little.
    bound[k + 1] = 1.001 * largest(c[0], c[1], c[2], bound[k]);
    if (!(bound[k + 1] <= 65536.0)) return SGEMM_ERR_INVALID_VALUE;
  }
  if (sizes != SGEMM_OK) return sizes;
  if (ldx > kMaxDim || ldy > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  const bool writes = batch > 0 && M > 0 && N > 0;
  if (writes) {
    if (!X || !Y || misaligned(X, size_of(typeX)) || misaligned(Y, size_of(typeY)) || !workspace ||
        misaligned(workspace, 16) || workspace_bytes < Layout(batch, M, N).total)
      return SGEMM_ERR_INVALID_VALUE;
  }
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  int cus = 0;
  const int rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);

  const Layout l(batch, M, N);
  if (l.is_short)
    return short_steps(l, batch, M, N, steps, sets, coefficients, eps, alpha, typeX, X, ldx,
                       strideX, typeY, Y, ldy, strideY, workspace, s);
  char *at = static_cast<char *>(workspace);
  auto take = [&](int64_t bytes) {
    char *const from = at;
    at += batch * bytes;
    return from;
  };
  auto matrix = [&](int rows, int cols) {
    const int64_t bytes = sgemm::split_bytes(rows, cols);
    return sgemm::SplitMatrix{take(bytes), rows, cols, bytes};
  };
  const sgemm::SplitMatrix z = matrix(l.m, l.n), S = matrix(l.m, l.m), P = matrix(l.m, l.m);
  sgemm::SplitMatrix zt[2] = {matrix(l.n, l.m), matrix(l.n, l.m)};
  const sgemm::SplitMatrix z_floats = matrix(l.n, l.m), s_floats = matrix(l.m, l.m), none{nullptr, 0, 0, 0};
  const bool tall = M > N;

  sgemm::OrthoSizesArgs in;
  in.M = (int)M;
  in.N = (int)N;
  in.X = X;
  in.ldx = ldx;
  in.strideX = strideX;
  in.eps = eps;
  in.band = sgemm::sizes_band(M, N);
  in.bands = sgemm::sizes_bands(M, N);
  in.runs = sgemm::sizes_runs(N);
  in.summed = in.bands + in.runs > sgemm::kMostSizeParts;
  in.parts = reinterpret_cast<double *>(take(8 * l.parts));
  in.scale = reinterpret_cast<double *>(take(8));
  in.row_parts = reinterpret_cast<unsigned *>(take(l.row_parts));
  in.col_parts = reinterpret_cast<unsigned *>(take(l.col_parts));
  in.rows = reinterpret_cast<unsigned *>(take(l.rows));
  in.cols = reinterpret_cast<unsigned *>(take(l.cols));
  in.again = (int)((steps - 1) / kLookAgain);
  const bool x_bf16 = typeX == SGEMM_TYPE_BF16, y_bf16 = typeY == SGEMM_TYPE_BF16;

  // Z's rows and columns: their largest magnitudes when they were last looked at, `look`,
  // times the root of their length bound their norms (2^of_rows, 2^of_cols times the power
  // of two above the magnitude), and `growth` what these have become since.
  unsigned *const tops_m = tall ? in.cols : in.rows, *const tops_n = tall ? in.rows : in.cols;
  const int of_rows = exponent_of(sqrt((double)l.n)), of_cols = exponent_of(sqrt((double)l.m));
  int look = 0;
  double growth = 1;
  // The scale of Z's rows (or columns) before step k, and of what is as much larger as
  // 2^more.
  auto scale_of = [&](bool rows, int64_t k, int more) {
    const int add = (rows ? of_rows : of_cols) + exponent_of(growth) - 126 + more;
    return sgemm::RowScale{
        rows ? tops_m + look * batch * l.m : tops_n + look * batch * l.n, add,
        exponent_of(bound[k]) + more};
  };
  sgemm::OrthoSplitArgs split;
  split.x = in;
  sgemm::RowScale z_scale = scale_of(true, 0, 0), zt_scale = scale_of(false, 0, 0);  // as held
  split.row_scale = tall ? zt_scale : z_scale;
  split.col_scale = tall ? z_scale : zt_scale;
  split.rows = tall ? zt[0] : z;
  split.cols = tall ? z : zt[0];
  split.floats = z_floats;
  split.floats_turned = !tall;
  hipError_t err = sgemm::launch_ortho_sizes(in, x_bf16, (int)batch, s);
  if (err == hipSuccess) err = sgemm::launch_ortho_split(split, x_bf16, (int)batch, s);
  for (int64_t k = 0; k < steps && err == hipSuccess; ++k) {
    const float *c = coefficients + (sets == 1 ? 0 : 3 * k);
    const double top = bound[k] * bound[k];
    // A row of S is at most the largest singular value times Z's row, one of P at most
    // that times |b| + |c| |S|.
    const int more_s = exponent_of(bound[k]);
    const int more_p = exponent_of(bound[k] * (fabs(c[1]) + fabs(c[2]) * top));
    const bool last = k + 1 == steps;
    sgemm::OrthoProductArgs p{};
    p.e = p.d_t = p.f_t = none;
    // S = Z Z^T
    p.a = p.b = z;
    p.a_scale = p.b_scale = z_scale;
    p.f1 = 1.f;
    p.d = S;
    p.d_scale = p.d_t_scale = scale_of(true, k, more_s);
    p.f_t = s_floats;
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // P = b S + c S S
    p.a = p.b = S;
    p.a_scale = p.b_scale = p.d_scale;
    p.e = s_floats;
    p.f_t = none;
    p.f1 = c[2];
    p.f2 = c[1];
    p.d = P;
    p.d_scale = p.d_t_scale = scale_of(true, k, more_p);
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // a Z + P Z
    p.a = P;
    p.b = zt[k % 2];
    p.a_scale = p.d_scale;
    p.b_scale = zt_scale;
    p.e = z_floats;
    p.f1 = 1.f;
    p.f2 = c[0];
    if (last) {
      p.d = none;
      p.d_t_scale = p.b_scale;  // read, but not used, as d_scale is
      p.Y = Y;
      p.ldy = ldy;
      p.strideY = strideY;
      p.y_transposed = tall;
      p.alpha = alpha;
    } else {
      growth = fmin(growth * 1.001 * largest_growth(c[0], c[1], c[2], top), 1e300);
      p.d = z;
      p.d_scale = scale_of(true, k + 1, 0);
      p.d_t = zt[1 - k % 2];
      p.d_t_scale = scale_of(false, k + 1, 0);
      p.f_t = z_floats;
    }
    err = sgemm::launch_ortho_product(p, false, y_bf16, (int)batch, cus, s);
    z_scale = p.d_scale;
    zt_scale = p.d_t_scale;
    if (!last && (k + 1) % kLookAgain == 0 && err == hipSuccess) {
      ++look;
      growth = 1;
      err = sgemm::launch_ortho_look(z_floats, tops_n + look * batch * l.n,
                                     tops_m + look * batch * l.m, (int)batch, s);
    }
  }
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // extern "C"
