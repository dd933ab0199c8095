// api_int8.hip -- the C interface declared in include/sgemm_int8.h: argument
// checks, the workspace's layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "api_internal.hpp"
#include "grouped_map.hpp"
#include "int8.hpp"
#include "sgemm_grouped.h"
#include "sgemm_int8.h"

namespace {

using sgemm_api::kMaxDim;
using sgemm_api::kMaxWorkItems;

constexpr int64_t kSlice = sgemm::kSliceRow;
constexpr int64_t kMaxK = (int64_t(1) << 17) - 1;
constexpr int64_t kMaxPitch = int64_t(1) << 22;  // offsets in a tile of 256 rows: below 2^30
constexpr int64_t kMaxLdc = int64_t(1) << 27;    // offsets in 8 rows of C: below 4 GiB

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
int64_t kp(int64_t K) { return sgemm::int8_kp(K); }
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_sizes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0) return SGEMM_ERR_INVALID_VALUE;
  return rows > kMaxDim || K > kMaxK ? SGEMM_ERR_TOO_LARGE : SGEMM_OK;
}

// A work-group of 256 for each row at the most.
bool cast_fits(int64_t rows) { return rows <= kMaxWorkItems / 256; }

bool bad_pitch(int64_t ld, int64_t K) { return ld < kp(K) || ld % 16 != 0; }

// The codes come first in a workspace, slice by slice, the scales after them.
int64_t codes_bytes(int64_t rows, int64_t K) { return rows * kp(K); }

// Both product entry points; groups < 0: not grouped.
int run(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
        int64_t lda, const float *scalesA, const void *B, int64_t ldb, const float *scalesB,
        float beta, int typeC, void *C, int64_t ldc, const int64_t *offsets, void *workspace,
        int64_t workspace_bytes, void *stream) {
  const bool grouped = groups >= 0;
  const bool held = typeA == SGEMM_TYPE_INT8;
  if ((!held && typeA != SGEMM_TYPE_F32 && typeA != SGEMM_TYPE_BF16) ||
      (typeC != SGEMM_TYPE_F32 && typeC != SGEMM_TYPE_BF16))
    return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_VALUE;
  if (ldc < (N > 1 ? N : 1) || (held ? bad_pitch(lda, K) : lda < (K > 1 ? K : 1)) ||
      bad_pitch(ldb, K))
    return SGEMM_ERR_INVALID_VALUE;
  const int64_t b_groups = grouped ? groups : 1;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK || lda > kMaxDim || (held && lda >= kMaxPitch) ||
      ldb >= kMaxPitch || ldc >= kMaxLdc || b_groups > SGEMM_GROUPED_MAX_GROUPS)
    return SGEMM_ERR_TOO_LARGE;
  const bool writes = M > 0 && N > 0 && b_groups > 0;
  const bool reads_ab = writes && K > 0 && alpha != 0.f;
  // Work-items for a block of 16 x 16: 512 at the most.
  const int64_t rows = grouped ? sgemm::group_tile_rows(M, groups, 16) : tiles(M, 16);
  if (rows > kMaxWorkItems / 512 / (N ? tiles(N, 16) : 1)) return SGEMM_ERR_TOO_LARGE;
  if (reads_ab && !held && !cast_fits(M)) return SGEMM_ERR_TOO_LARGE;
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
          misaligned(workspace, 16) || workspace_bytes < sgemm_int8_workspace_size(typeA, M, K))
        return SGEMM_ERR_INVALID_VALUE;
    }
  }
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  int cus = 0;
  const int rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);

  sgemm::Int8Args p;
  p.M = (int)M;
  p.N = (int)N;
  p.K = reads_ab ? (int)K : 0;
  p.groups = (int)b_groups;
  p.alpha = reads_ab ? alpha : 0.f;  // an empty sum is 0, whatever alpha is
  p.beta = beta;
  p.a = {static_cast<const char *>(A), scalesA, lda, kSlice};
  p.b = {static_cast<const char *>(B), scalesB, ldb, kSlice};
  p.C = C;
  p.ldc = ldc;
  p.offsets = grouped ? offsets : nullptr;
  hipError_t err = hipSuccess;
  int a_type = SGEMM_TYPE_INT8;
  if (reads_ab && !held) {
    if (sgemm::int8_casts(p, cus)) {
      a_type = typeA;
    } else {
      char *codes = static_cast<char *>(workspace);
      float *scales = reinterpret_cast<float *>(codes + codes_bytes(M, K));
      err = sgemm::launch_int8_quantize(false, typeA == SGEMM_TYPE_BF16,
                                        {(int)M, (int)K, lda, A, codes, kSlice, M * kSlice, scales},
                                        s);
      p.a = {codes, scales, kSlice, M * kSlice};
    }
  }
  if (err == hipSuccess)
    err = sgemm::launch_int8_product(p, a_type, typeC == SGEMM_TYPE_BF16, cus, s);
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int64_t sgemm_int8_codes_size(int64_t rows, int64_t K) {
  const int rc = check_sizes(rows, K);
  return rc != SGEMM_OK ? rc : codes_bytes(rows, K);
}

int64_t sgemm_int8_workspace_size(int typeA, int64_t M, int64_t K) {
  if (typeA != SGEMM_TYPE_F32 && typeA != SGEMM_TYPE_BF16 && typeA != SGEMM_TYPE_INT8)
    return SGEMM_ERR_INVALID_VALUE;
  const int rc = check_sizes(M, K);
  if (rc != SGEMM_OK) return rc;
  return typeA == SGEMM_TYPE_INT8 ? 0 : codes_bytes(M, K) + 4 * M;
}

int sgemm_int8_quantize(int trans, int64_t rows, int64_t K, int type, const void *X, int64_t ldx,
                        void *codes, int64_t ldq, float *scales, void *stream) {
  if ((trans != 0 && trans != 1) || (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16))
    return SGEMM_ERR_INVALID_VALUE;
  int rc = check_sizes(rows, K);
  if (rc == SGEMM_ERR_INVALID_VALUE) return rc;
  const int64_t cols = trans ? rows : K;
  if (ldx < (cols > 1 ? cols : 1) || bad_pitch(ldq, K)) return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (ldx > kMaxDim || ldq > kMaxDim || !cast_fits(rows)) return SGEMM_ERR_TOO_LARGE;
  if (rows > 0 && K > 0 &&
      (!X || !codes || !scales || misaligned(X, type == SGEMM_TYPE_F32 ? 4 : 2) ||
       misaligned(codes, 16) || misaligned(scales, 4)))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (rows == 0 || K == 0) return SGEMM_OK;
  int cus = 0;
  rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  const hipError_t err = sgemm::launch_int8_quantize(
      trans != 0, type == SGEMM_TYPE_BF16,
      {(int)rows, (int)K, ldx, X, static_cast<char *>(codes), ldq, kSlice, scales},
      reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

int sgemm_run_int8(int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
                   int64_t lda, const float *scalesA, const void *B, int64_t ldb,
                   const float *scalesB, float beta, int typeC, void *C, int64_t ldc,
                   void *workspace, int64_t workspace_bytes, void *stream) {
  return run(-1, M, N, K, alpha, typeA, A, lda, scalesA, B, ldb, scalesB, beta, typeC, C, ldc,
             nullptr, workspace, workspace_bytes, stream);
}

int sgemm_run_int8_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                           int typeA, const void *A, int64_t lda, const float *scalesA,
                           const void *B, int64_t ldb, const float *scalesB, float beta,
                           int typeC, void *C, int64_t ldc, const int64_t *offsets,
                           void *workspace, int64_t workspace_bytes, void *stream) {
  if (groups < 0) return SGEMM_ERR_INVALID_VALUE;
  return run(groups, M, N, K, alpha, typeA, A, lda, scalesA, B, ldb, scalesB, beta, typeC, C, ldc,
             offsets, workspace, workspace_bytes, stream);
}

}  // extern "C"
