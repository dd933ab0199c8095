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

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool bad_type(int type) { return type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16; }
unsigned size_of(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// The workspace: Z, P, Z transposed, S, Z transposed again (a step reads one and writes the
// other).  The exponents of the rows' and columns' norms, twice (as Z is held, and as it was
// last looked at), have an end of S's room, the one away from the transposed Z that the
// step writes: S, until then, reaches into that, and the step's last launch moves the
// exponents to the other end.  (All of S there, 16 of 256 x 256 took 10.2 us for 7.9.)
// Before, the parts of the norms and sizes are in the second transposed Z.  Short matrices:
// the parts of the norms, and Z and the parts of S twice.
struct Layout {
  int m, n;
  int64_t z, zt, s;     // bytes of a matrix
  int64_t parts;        // of a norm
  int64_t total;
  int shared;           // 2^shared columns of Z share an exponent, so that there is room
  // Where m is short: Z and S's parts, twice each.
  bool is_short;
  int64_t short_z, short_parts;
  Layout(int64_t batch, int64_t M, int64_t N) {
    m = (int)(M < N ? M : N);
    n = (int)(M < N ? N : M);
    z = sgemm::split_bytes(m, n);
    zt = sgemm::split_bytes(n, m);
    s = sgemm::split_bytes(m, m);
    parts = tiles(M * tiles(N, sgemm::kNormRun), 16);
    if (parts > sgemm::kNormParts) parts = sgemm::kNormParts;
    is_short = m <= sgemm::kShort;
    shared = 0;
    while (!is_short && 2 * norms(1) > s) ++shared;  // ends: 65 rows have 24960 bytes
    short_z = 4 * (int64_t)m * n;
    short_parts = 4 * (int64_t)m * m * sgemm::short_slabs(n);
    total = batch * (8 * parts + (is_short ? 2 * (short_z + short_parts) : z + 2 * zt + 2 * s));
  }
  int64_t columns() const { return (int64_t)((n - 1) >> shared) + 1; }
  // Bytes of the exponents, and of the scale.
  int64_t norms(int64_t batch) const { return tiles(batch * (8 + 2 * (m + columns())), 128) * 128; }
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
  const sgemm::SplitMatrix z = matrix(l.m, l.n), P = matrix(l.m, l.m), zt0 = matrix(l.n, l.m),
                           room = matrix(l.m, l.m), zt1 = matrix(l.n, l.m);
  const sgemm::SplitMatrix zt[2] = {zt0, zt1}, none{nullptr, 0, 0, 0};
  const bool tall = M > N;
  const int64_t norms = l.norms(batch);
  // Where step k has the exponents.
  auto norms_at = [&](int64_t k) { return k % 2 ? room.at + batch * l.s - norms : room.at; };

  // Z's rows and columns by exponents of their norms: those of `set`, which are from when
  // they were looked at last, and what the steps since can have made of them; and at most
  // those of the whole matrix.
  struct Range {
    int set, grown, most;
    Range with(int more) const { return {set, grown + more, most + more}; }
  };
  auto norms_of = [&](int64_t k, int set, bool rows) {
    return reinterpret_cast<signed char *>(norms_at(k)) +
           batch * (8 + set * (l.m + l.columns()) + (rows ? 0 : l.m));
  };
  auto scale_of = [&](int64_t k, const Range &x, bool rows) {
    return sgemm::RowScale{norms_of(k, x.set, rows), rows ? l.m : (int)l.columns(),
                           rows ? 0 : l.shared, x.grown, x.most};
  };
  int set = 0;
  double growth = 1;
  auto range = [&](int64_t k) { return Range{set, exponent_of(growth), exponent_of(bound[k])}; };
  Range held = range(0);  // Z, as it is held

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
  in.parts = reinterpret_cast<double *>(zt1.at);
  in.row_parts = reinterpret_cast<unsigned *>(in.parts + batch * in.bands * in.runs);
  in.col_parts = in.row_parts + batch * in.runs * M;
  in.summed = l.shared > 0 || in.bands + in.runs > sgemm::kMostSizeParts;
  in.scale = reinterpret_cast<double *>(norms_at(0));
  in.rows = norms_of(0, 0, !tall);
  in.cols = norms_of(0, 0, tall);
  in.row_shift = tall ? l.shared : 0;
  in.col_shift = tall ? 0 : l.shared;
  in.row_length = exponent_of(sqrt((double)N));
  in.col_length = exponent_of(sqrt((double)M));
  const bool x_bf16 = typeX == SGEMM_TYPE_BF16, y_bf16 = typeY == SGEMM_TYPE_BF16;
  sgemm::OrthoSplitArgs split;
  split.x = in;
  split.row_scale = scale_of(0, held, !tall);
  split.col_scale = scale_of(0, held, tall);
  split.rows = tall ? zt0 : z;
  split.cols = tall ? z : zt0;
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
    const sgemm::SplitMatrix S{k % 2 ? room.at - norms : room.at + norms, l.m, l.m, l.s};
    sgemm::OrthoProductArgs p{};
    p.e = p.e_t = p.d_t = none;
    // S = Z Z^T
    p.a = p.b = z;
    p.a_scale = p.b_scale = p.e_scale = scale_of(k, held, true);
    p.f1 = 1.f;
    p.d = S;
    p.d_scale = p.d_t_scale = scale_of(k, range(k).with(more_s), true);
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // P = b S + c S S
    p.a = p.b = p.e = p.e_t = S;
    p.a_scale = p.b_scale = p.e_scale = p.d_scale;
    p.f1 = c[2];
    p.f2 = c[1];
    p.d = P;
    p.d_scale = p.d_t_scale = scale_of(k, range(k).with(more_p), true);
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // a Z + P Z
    p.a = P;
    p.b = p.e_t = zt[k % 2];
    p.e = z;
    p.a_scale = p.d_scale;
    p.b_scale = scale_of(k, held, false);
    p.e_scale = scale_of(k, held, true);
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
      held = range(k + 1);
      p.d = z;
      p.d_scale = scale_of(k, held, true);
      p.d_t = zt[1 - k % 2];
      p.d_t_scale = scale_of(k, held, false);
      p.move_from = norms_at(k);
      p.move_to = norms_at(k + 1);
      p.moves = (unsigned)(norms / 16);  // below 2^27
    }
    err = sgemm::launch_ortho_product(p, false, y_bf16, (int)batch, cus, s);
    if (!last && (k + 1) % kLookAgain == 0 && err == hipSuccess) {
      set = 1 - set;
      growth = 1;
      sgemm::OrthoSizesArgs again{};
      again.M = l.m;
      again.N = l.n;
      again.bands = again.runs = 1;
      again.row_parts = reinterpret_cast<unsigned *>(zt[k % 2].at);
      again.col_parts = again.row_parts + batch * l.m;
      again.rows = norms_of(k + 1, set, true);
      again.cols = norms_of(k + 1, set, false);
      again.col_shift = l.shared;
      again.row_length = exponent_of(sqrt((double)l.n));
      again.col_length = exponent_of(sqrt((double)l.m));
      err = sgemm::launch_ortho_look(again, z, scale_of(k + 1, held, true), (int)batch, s);
    }
  }
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // extern "C"
