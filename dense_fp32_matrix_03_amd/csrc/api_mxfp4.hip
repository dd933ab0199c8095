// api_mxfp4.hip -- the C interface declared in include/sgemm_mxfp4.h: argument
// checks, the workspace's layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "api_internal.hpp"
#include "grouped_map.hpp"
#include "mxfp4.hpp"
#include "sgemm_grouped.h"
#include "sgemm_mxfp4.h"

namespace {

using sgemm_api::kMaxDim;
using sgemm_api::kMaxWorkItems;

constexpr int64_t kMaxK = int64_t(1) << 21;
constexpr int64_t kMaxLdc = int64_t(1) << 27;  // offsets in 8 rows of C: below 4 GiB

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
int64_t kp(int64_t K) { return sgemm::mxfp4_kp(K); }
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_sizes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0) return SGEMM_ERR_INVALID_VALUE;
  return rows > kMaxDim || K > kMaxK ? SGEMM_ERR_TOO_LARGE : SGEMM_OK;
}

// Work-groups of a cast: 32 rows by 128 k each at the least.
bool cast_fits(int64_t rows, int64_t K) {
  return tiles(rows, 32) * (kp(K) / 128) <= kMaxWorkItems / 256;
}

int check_cast(int trans, int64_t rows, int64_t K, int type, const void *X, int64_t ldx,
               const void *codes, const void *scales, int64_t lds) {
  if ((trans != 0 && trans != 1) || (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16))
    return SGEMM_ERR_INVALID_VALUE;
  const int rc = check_sizes(rows, K);
  if (rc == SGEMM_ERR_INVALID_VALUE) return rc;
  const int64_t cols = trans ? rows : K;
  if (ldx < (cols > 1 ? cols : 1) || lds < rows) return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (ldx > kMaxDim || lds > kMaxDim || !cast_fits(rows, K)) return SGEMM_ERR_TOO_LARGE;
  if (rows == 0 || K == 0) return SGEMM_OK;
  if (!X || !codes || !scales || misaligned(X, type == SGEMM_TYPE_F32 ? 4 : 2) ||
      misaligned(codes, 16) || misaligned(scales, 4))
    return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

sgemm::CastArgs cast_args(int64_t rows, int64_t K, const void *X, int64_t ldx, void *codes,
                          void *scales, int64_t lds) {
  sgemm::CastArgs p;
  p.rows = (int)rows;
  p.K = (int)K;
  p.ldx = ldx;
  p.granules = (int)(kp(K) / 128);
  p.lds = lds;
  p.X = X;
  p.codes = codes;
  p.scales = static_cast<unsigned *>(scales);
  return p;
}

// The codes come first in a workspace, the scales after them.
int64_t codes_bytes(int64_t rows, int64_t K) { return rows * (kp(K) / 2); }

// Both product entry points; groups < 0: not grouped.
int run(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
        int64_t lda, const void *scalesA, const void *B, const void *scalesB, int64_t ldsb,
        float beta, int typeC, void *C, int64_t ldc, const int64_t *offsets, void *workspace,
        int64_t workspace_bytes, void *stream) {
  const bool grouped = groups >= 0;
  const bool held = typeA == SGEMM_TYPE_MXFP4;
  if ((!held && typeA != SGEMM_TYPE_F32 && typeA != SGEMM_TYPE_BF16) ||
      (typeC != SGEMM_TYPE_F32 && typeC != SGEMM_TYPE_BF16))
    return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_VALUE;
  const int64_t b_groups = grouped ? groups : 1;
  const int64_t a_cols = held ? M : K;
  if (lda < (a_cols > 1 ? a_cols : 1) || ldc < (N > 1 ? N : 1)) return SGEMM_ERR_INVALID_VALUE;
  if ((__int128)b_groups * N > ldsb) return SGEMM_ERR_INVALID_VALUE;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK || lda > kMaxDim || ldsb > kMaxDim ||
      ldc >= kMaxLdc || b_groups > SGEMM_GROUPED_MAX_GROUPS)
    return SGEMM_ERR_TOO_LARGE;
  const bool writes = M > 0 && N > 0 && b_groups > 0;
  const bool reads_ab = writes && K > 0 && alpha != 0.f;
  // Work-items for a block of 16 x 16: 256 at the most, but 512 with eight waves to it.
  const int64_t block =
      !grouped && M <= 16 && sgemm::mxfp4_eight_sets(reads_ab ? K : 0) ? 512 : 256;
  const int64_t rows = grouped ? sgemm::group_tile_rows(M, groups, 16) : tiles(M, 16);
  if (rows > kMaxWorkItems / block / (N ? tiles(N, 16) : 1)) return SGEMM_ERR_TOO_LARGE;
  if (reads_ab && !held && !cast_fits(M, K)) return SGEMM_ERR_TOO_LARGE;
  if (writes && (!C || misaligned(C, typeC == SGEMM_TYPE_F32 ? 4 : 2) ||
                 (grouped && (!offsets || misaligned(offsets, 8)))))
    return SGEMM_ERR_INVALID_VALUE;
  if (reads_ab) {
    if (!A || !B || !scalesB || misaligned(B, 16) || misaligned(scalesB, 4))
      return SGEMM_ERR_INVALID_VALUE;
    if (held) {
      if (!scalesA || misaligned(A, 16) || misaligned(scalesA, 4)) return SGEMM_ERR_INVALID_VALUE;
    } else {
      if (misaligned(A, typeA == SGEMM_TYPE_F32 ? 4 : 2) || !workspace ||
          misaligned(workspace, 16) ||
          workspace_bytes < sgemm_mxfp4_workspace_size(typeA, M, K))
        return SGEMM_ERR_INVALID_VALUE;
    }
  }
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  int cus = 0;
  const int rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);

  sgemm::Mxfp4Args p;
  p.M = (int)M;
  p.N = (int)N;
  p.K = reads_ab ? (int)K : 0;
  p.groups = (int)b_groups;
  p.alpha = reads_ab ? alpha : 0.f;  // an empty sum is 0, whatever alpha is
  p.beta = beta;
  p.a = {static_cast<const unsigned char *>(A), static_cast<const unsigned *>(scalesA), lda};
  p.b = {static_cast<const unsigned char *>(B), static_cast<const unsigned *>(scalesB), ldsb};
  p.C = C;
  p.ldc = ldc;
  p.offsets = grouped ? offsets : nullptr;
  hipError_t err = hipSuccess;
  int a_type = SGEMM_TYPE_MXFP4;
  if (reads_ab && !held) {
    if (sgemm::mxfp4_casts(p, cus)) {
      a_type = typeA;
    } else {
      unsigned char *codes = static_cast<unsigned char *>(workspace);
      unsigned char *scales = codes + codes_bytes(M, K);
      err = sgemm::launch_mxfp4_quantize(false, typeA == SGEMM_TYPE_BF16,
                                         cast_args(M, K, A, lda, codes, scales, M), s);
      p.a = {codes, reinterpret_cast<unsigned *>(scales), (long)M};
    }
  }
  if (err == hipSuccess)
    err = sgemm::launch_mxfp4_product(p, a_type, typeC == SGEMM_TYPE_BF16, cus, s);
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int64_t sgemm_mxfp4_codes_size(int64_t rows, int64_t K) {
  const int rc = check_sizes(rows, K);
  return rc != SGEMM_OK ? rc : codes_bytes(rows, K);
}

int64_t sgemm_mxfp4_scales_size(int64_t rows, int64_t K) {
  const int rc = check_sizes(rows, K);
  return rc != SGEMM_OK ? rc : rows * (kp(K) / 32);
}

int64_t sgemm_mxfp4_workspace_size(int typeA, int64_t M, int64_t K) {
  if (typeA < SGEMM_TYPE_F32 || typeA > SGEMM_TYPE_MXFP4) return SGEMM_ERR_INVALID_VALUE;
  const int rc = check_sizes(M, K);
  if (rc != SGEMM_OK) return rc;
  return typeA == SGEMM_TYPE_MXFP4 ? 0 : codes_bytes(M, K) + M * (kp(K) / 32);
}

int sgemm_mxfp4_quantize(int trans, int64_t rows, int64_t K, int type, const void *X, int64_t ldx,
                         void *codes, void *scales, int64_t lds, void *stream) {
  int rc = check_cast(trans, rows, K, type, X, ldx, codes, scales, lds);
  if (rc != SGEMM_OK) return rc;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (rows == 0 || K == 0) return SGEMM_OK;
  int cus = 0;
  rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  const hipError_t err = sgemm::launch_mxfp4_quantize(
      trans != 0, type == SGEMM_TYPE_BF16, cast_args(rows, K, X, ldx, codes, scales, lds),
      reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

int sgemm_mxfp4_dequantize(int trans, int64_t rows, int64_t K, const void *codes,
                           const void *scales, int64_t lds, int type, void *X, int64_t ldx,
                           void *stream) {
  int rc = check_cast(trans, rows, K, type, X, ldx, codes, scales, lds);
  if (rc != SGEMM_OK) return rc;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (rows == 0 || K == 0) return SGEMM_OK;
  int cus = 0;
  rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  const hipError_t err = sgemm::launch_mxfp4_dequantize(
      trans != 0, type == SGEMM_TYPE_BF16,
      cast_args(rows, K, X, ldx, const_cast<void *>(codes), const_cast<void *>(scales), lds),
      reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

int sgemm_run_mxfp4(int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
                    int64_t lda, const void *scalesA, const void *B, const void *scalesB,
                    int64_t ldsb, float beta, int typeC, void *C, int64_t ldc, void *workspace,
                    int64_t workspace_bytes, void *stream) {
  return run(-1, M, N, K, alpha, typeA, A, lda, scalesA, B, scalesB, ldsb, beta, typeC, C, ldc,
             nullptr, workspace, workspace_bytes, stream);
}

int sgemm_run_mxfp4_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                            int typeA, const void *A, int64_t lda, const void *scalesA,
                            const void *B, const void *scalesB, int64_t ldsb, float beta,
                            int typeC, void *C, int64_t ldc, const int64_t *offsets,
                            void *workspace, int64_t workspace_bytes, void *stream) {
  if (groups < 0) return SGEMM_ERR_INVALID_VALUE;
  return run(groups, M, N, K, alpha, typeA, A, lda, scalesA, B, scalesB, ldsb, beta, typeC, C,
             ldc, offsets, workspace, workspace_bytes, stream);
}

}  // extern "C"
