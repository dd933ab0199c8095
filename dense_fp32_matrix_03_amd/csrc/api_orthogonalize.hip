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

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool bad_type(int type) { return type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16; }
unsigned size_of(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// The workspace: Z, Z transposed twice (a step reads one and writes the other), S
// and P of every matrix, and the parts of the norms.  Short matrices: the parts of the
// norms, and Z and the parts of S twice.
struct Layout {
  int m, n;
  int64_t z, zt, s;     // bytes of a matrix
  int64_t parts;        // of a norm
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
    parts = tiles(M * tiles(N, sgemm::kNormRun), 16);
    if (parts > sgemm::kNormParts) parts = sgemm::kNormParts;
    is_short = m <= sgemm::kShort;
    short_z = 4 * (int64_t)m * n;
    short_parts = 4 * (int64_t)m * m * sgemm::short_slabs(n);
    total = batch * (8 * parts + (is_short ? 2 * (short_z + short_parts) : z + 2 * zt + 2 * s));
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

// The power of two by which a matrix with no element above `bound` is held: the
// largest stays below 2^15, half of what half precision holds.
int shift_for(double bound) {
  int e;
  frexp(fmax(bound * 1.02, ldexp(1.0, -60)), &e);  // below 2^e
  return 15 - e;
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
  auto matrix = [&](int rows, int cols) {
    const sgemm::SplitMatrix x{at, rows, cols, sgemm::split_bytes(rows, cols)};
    at += batch * x.stride;
    return x;
  };
  const sgemm::SplitMatrix z = matrix(l.m, l.n), S = matrix(l.m, l.m), P = matrix(l.m, l.m);
  sgemm::SplitMatrix zt[2] = {matrix(l.n, l.m), matrix(l.n, l.m)};
  const sgemm::SplitMatrix none{nullptr, 0, 0, 0};
  const bool tall = M > N;

  sgemm::OrthoSplitArgs in;
  in.x = {(int)M, (int)N, X, ldx, strideX, reinterpret_cast<double *>(at), (int)l.parts};
  in.eps = eps;
  int shift = shift_for(bound[0]);
  in.shift = shift;
  in.rows = tall ? zt[0] : z;
  in.cols = tall ? z : zt[0];
  const bool x_bf16 = typeX == SGEMM_TYPE_BF16, y_bf16 = typeY == SGEMM_TYPE_BF16;
  hipError_t err = sgemm::launch_ortho_norm(in.x, x_bf16, (int)batch, s);
  if (err == hipSuccess) err = sgemm::launch_ortho_split(in, x_bf16, (int)batch, s);
  for (int64_t k = 0; k < steps && err == hipSuccess; ++k) {
    const float *c = coefficients + (sets == 1 ? 0 : 3 * k);
    const double top = bound[k] * bound[k];
    const int shift_s = shift_for(top);
    const int shift_p = shift_for(fabs(c[1]) * top + fabs(c[2]) * top * top);
    const bool last = k + 1 == steps;
    const int shift_y = last ? 0 : shift_for(bound[k + 1]);
    const double out = last ? alpha : 1.0;
    sgemm::OrthoProductArgs p;
    p.Y = nullptr;
    p.ldy = p.strideY = 0;
    p.y_transposed = false;
    // S = Z Z^T
    p.a = p.b = z;
    p.e_t = none;
    p.f1 = (float)ldexp(1.0, shift_s - 2 * shift);
    p.f2 = 0.f;
    p.d = S;
    p.d_t = none;
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // P = b S + c S S
    p.a = p.b = p.e_t = S;
    p.f1 = (float)(c[2] * ldexp(1.0, shift_p - 2 * shift_s));
    p.f2 = (float)(c[1] * ldexp(1.0, shift_p - shift_s));
    p.d = P;
    err = sgemm::launch_ortho_product(p, true, false, (int)batch, cus, s);
    if (err != hipSuccess) break;
    // a Z + P Z
    p.a = P;
    p.b = p.e_t = zt[k % 2];
    p.f1 = (float)(out * ldexp(1.0, shift_y - shift_p - shift));
    p.f2 = (float)(out * c[0] * ldexp(1.0, shift_y - shift));
    p.d = last ? none : z;
    p.d_t = last ? none : zt[1 - k % 2];
    if (last) {
      p.Y = Y;
      p.ldy = ldy;
      p.strideY = strideY;
      p.y_transposed = tall;
    }
    err = sgemm::launch_ortho_product(p, false, y_bf16, (int)batch, cus, s);
    shift = shift_y;
  }
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // extern "C"
