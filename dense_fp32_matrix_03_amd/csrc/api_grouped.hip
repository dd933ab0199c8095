// api_grouped.hip -- the C interface declared in include/sgemm_grouped.h:
// argument checks and the launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "api_internal.hpp"
#include "grouped.hpp"
#include "grouped_map.hpp"
#include "sgemm_grouped.h"

namespace {

using sgemm_api::kMaxDim;
using sgemm_api::kMaxWorkItems;

constexpr int64_t kMaxLd = int64_t(1) << 22;   // offsets in a tile of 128 rows: below 2 GiB
constexpr int64_t kMaxK = int64_t(1) << 30;    // rows of grouped_k: positions in K stay below 2^31
constexpr int64_t kMaxLdc = int64_t(1) << 27;  // offsets in 8 rows of C: below 4 GiB

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// The checks that the two forms share; a_cols, b_cols: stored widths.
int check(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t a_cols, int64_t lda,
          int64_t b_cols, int64_t ldb, int64_t ldc) {
  if (groups < 0 || M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_VALUE;
  if (lda < (a_cols > 1 ? a_cols : 1) || ldb < (b_cols > 1 ? b_cols : 1) || ldc < (N > 1 ? N : 1))
    return SGEMM_ERR_INVALID_VALUE;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || ldc >= kMaxLdc ||
      groups > SGEMM_GROUPED_MAX_GROUPS)
    return SGEMM_ERR_TOO_LARGE;
  return SGEMM_OK;
}

bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

int sgemm_run_grouped(int transB, int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                      const float *A, int64_t lda, const float *B, int64_t ldb, int64_t strideB,
                      float beta, float *C, int64_t ldc, const int64_t *offsets, void *stream) {
  if (transB != 0 && transB != 1) return SGEMM_ERR_INVALID_VALUE;
  int rc = check(groups, M, N, K, K, lda, transB ? K : N, ldb, ldc);
  if (rc == SGEMM_ERR_INVALID_VALUE || strideB < 0) return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (sgemm::group_tile_rows(M, groups, 32) > kMaxWorkItems / 256 / (N ? tiles(N, 32) : 1))
    return SGEMM_ERR_TOO_LARGE;
  const bool writes = groups > 0 && M > 0 && N > 0, reads_ab = writes && K > 0 && alpha != 0.f;
  if (reads_ab && (lda >= kMaxLd || ldb >= kMaxLd)) return SGEMM_ERR_TOO_LARGE;
  if (writes && (!C || !offsets || misaligned(C, 4) || misaligned(offsets, 8)))
    return SGEMM_ERR_INVALID_VALUE;
  if (reads_ab && (!A || !B || misaligned(A, 4) || misaligned(B, 4))) return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  int cus = 0;
  rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  sgemm::GroupedArgs p{(int)M, (int)N, (int)K, (int)groups, alpha, beta, A,      lda,
                       B,      ldb,    strideB, C,          ldc,   0,    offsets};
  const hipError_t err =
      sgemm::launch_grouped_rows(p, transB != 0, cus, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

int sgemm_run_grouped_k(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                        const float *A, int64_t lda, const float *B, int64_t ldb, float beta,
                        float *C, int64_t ldc, int64_t strideC, const int64_t *offsets,
                        void *stream) {
  int rc = check(groups, M, N, K, M, lda, N, ldb, ldc);
  if (rc == SGEMM_ERR_INVALID_VALUE || strideC < 0) return SGEMM_ERR_INVALID_VALUE;
  // Distinct groups write disjoint C matrices.
  if (groups > 1 && M > 0 && N > 0 && (__int128)(M - 1) * ldc + N > strideC)
    return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (K > kMaxK) return SGEMM_ERR_TOO_LARGE;
  if (groups > 0 && tiles(M, 32) * tiles(N, 32) > kMaxWorkItems / 256 / groups)
    return SGEMM_ERR_TOO_LARGE;
  const bool writes = groups > 0 && M > 0 && N > 0, reads_ab = writes && K > 0 && alpha != 0.f;
  if (reads_ab && (lda >= kMaxLd || ldb >= kMaxLd)) return SGEMM_ERR_TOO_LARGE;
  if (writes && (!C || !offsets || misaligned(C, 4) || misaligned(offsets, 8)))
    return SGEMM_ERR_INVALID_VALUE;
  if (reads_ab && (!A || !B || misaligned(A, 4) || misaligned(B, 4))) return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  int cus = 0;
  rc = sgemm_api::current_device_cus(&cus);
  if (rc != SGEMM_OK) return rc;
  sgemm::GroupedArgs p{(int)M, (int)N, (int)K, (int)groups, alpha, beta, A,       lda,
                       B,      ldb,    0,      C,           ldc,   strideC, offsets};
  const hipError_t err =
      sgemm::launch_grouped_k(p, cus, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // extern "C"
