// api_route.hip -- the C interface declared in include/sgemm_route.h: argument
// checks and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "api_internal.hpp"
#include "route.hpp"
#include "sgemm_grouped.h"
#include "sgemm_route.h"

namespace {

using sgemm_api::kMaxDim;
using sgemm_api::kMaxWorkItems;

bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool bad_type(int type) { return type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16; }
unsigned size_of(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }
bool bad_pointer(const void *p, unsigned to) { return !p || misaligned(p, to); }
bool bad_flag(int f) { return f != 0 && f != 1; }

// Whether the library can launch: the last checks of every call.
int launchable() {
  int cus = 0;
  return sgemm_api::current_device_cus(&cus);
}
int status(hipError_t err) { return err == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }
hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

// The checks that sgemm_route and its gradient share.
int check_route(int64_t tokens, int64_t experts, int64_t topk, int score, int type, int64_t ldl,
                int renormalize) {
  if ((score != SGEMM_SCORE_SOFTMAX && score != SGEMM_SCORE_SIGMOID) || bad_type(type) ||
      bad_flag(renormalize) || tokens < 0 || experts < 1 || topk < 1 || topk > experts ||
      topk > SGEMM_ROUTE_MAX_TOPK || ldl < experts)
    return SGEMM_ERR_INVALID_VALUE;
  if (experts > SGEMM_ROUTE_MAX_EXPERTS || tokens > kMaxWorkItems / 64 - 4 ||
      tokens * topk > kMaxDim || ldl > kMaxDim)
    return SGEMM_ERR_TOO_LARGE;
  return SGEMM_OK;
}

// The checks that the calls that move rows share; rows: those that a wave has
// pieces of.
int check_rows(int64_t rows, int64_t units, int64_t N, int type, int64_t ldx, int64_t ldy) {
  if (rows > kMaxDim || N > kMaxDim || ldx > kMaxDim || ldy > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  const int64_t piece = sgemm::kRowPiece / size_of(type);
  const int64_t pieces = N > 0 ? (N + piece - 1) / piece : 1;
  return units > (kMaxWorkItems / 64 - 4) / pieces ? SGEMM_ERR_TOO_LARGE : SGEMM_OK;
}

int pieces_of(int64_t N, int type) {
  const int64_t piece = sgemm::kRowPiece / size_of(type);
  return (int)((N + piece - 1) / piece);
}

}  // namespace

extern "C" {

int sgemm_route(int64_t tokens, int64_t experts, int64_t topk, int score, int type,
                const void *logits, int64_t ldl, const float *bias, int64_t groups,
                int64_t topk_groups, int64_t group_top, int renormalize, float scale,
                int32_t *picks, float *weights, void *stream) {
  int rc = check_route(tokens, experts, topk, score, type, ldl, renormalize);
  if (rc == SGEMM_ERR_INVALID_VALUE || groups < 1 || groups > experts || experts % groups != 0 ||
      topk_groups < 1 || topk_groups > groups || (group_top != 1 && group_top != 2))
    return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (groups > SGEMM_ROUTE_MAX_GROUPS) return SGEMM_ERR_TOO_LARGE;
  if (tokens > 0 && (bad_pointer(logits, size_of(type)) || bad_pointer(picks, 4) ||
                     bad_pointer(weights, 4) || misaligned(bias, 4)))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (tokens == 0) return SGEMM_OK;
  if ((rc = launchable()) != SGEMM_OK) return rc;
  int share = 64;
  while (share * groups > 64) share /= 2;
  const sgemm::RouteArgs p{(int)tokens, (int)experts, (int)topk, score == SGEMM_SCORE_SIGMOID,
                           renormalize != 0, logits, ldl, bias, (int)groups, (int)topk_groups,
                           (int)group_top, scale, picks, weights,
                           sgemm::make_fast_div((int)(experts / groups)), share};
  return status(sgemm::launch_route(p, type == SGEMM_TYPE_BF16, stream_of(stream)));
}

int sgemm_route_backward(int64_t tokens, int64_t experts, int64_t topk, int score, int type,
                         const void *logits, int64_t ldl, int renormalize, float scale,
                         const int32_t *picks, const float *dweights, void *dlogits, int64_t ldd,
                         void *stream) {
  int rc = check_route(tokens, experts, topk, score, type, ldl, renormalize);
  if (rc == SGEMM_ERR_INVALID_VALUE || ldd < experts) return SGEMM_ERR_INVALID_VALUE;
  if (rc != SGEMM_OK) return rc;
  if (ldd > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  if (tokens > 0 && (bad_pointer(logits, size_of(type)) || bad_pointer(picks, 4) ||
                     bad_pointer(dweights, 4) || bad_pointer(dlogits, size_of(type))))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (tokens == 0) return SGEMM_OK;
  if ((rc = launchable()) != SGEMM_OK) return rc;
  const sgemm::RouteBackArgs p{(int)tokens, (int)experts, (int)topk, score == SGEMM_SCORE_SIGMOID,
                               renormalize != 0, logits, ldl, scale, picks, dweights, dlogits, ldd};
  return status(sgemm::launch_route_backward(p, type == SGEMM_TYPE_BF16, stream_of(stream)));
}

int64_t sgemm_route_plan_workspace_size(int64_t pairs, int64_t groups) {
  if (pairs < 0 || groups < 0) return SGEMM_ERR_INVALID_VALUE;
  if (pairs > kMaxDim || groups > SGEMM_GROUPED_MAX_GROUPS) return SGEMM_ERR_TOO_LARGE;
  const int64_t chunks = sgemm::plan_chunks(pairs);
  return chunks > 1 ? chunks * groups * 4 : 0;
}

int sgemm_route_plan(int64_t pairs, int64_t first, int64_t groups, const int32_t *picks,
                     int64_t *offsets, int32_t *sources, int32_t *places, void *workspace,
                     int64_t workspace_bytes, void *stream) {
  const int64_t need = sgemm_route_plan_workspace_size(pairs, groups);
  if (need == SGEMM_ERR_INVALID_VALUE || first < 0) return SGEMM_ERR_INVALID_VALUE;
  if (need < 0) return (int)need;
  if (first > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  if (bad_pointer(offsets, 8)) return SGEMM_ERR_INVALID_VALUE;
  if (pairs > 0 && (bad_pointer(picks, 4) || bad_pointer(sources, 4) || bad_pointer(places, 4)))
    return SGEMM_ERR_INVALID_VALUE;
  if (need > 0 && (bad_pointer(workspace, 16) || workspace_bytes < need))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  const int rc = launchable();
  if (rc != SGEMM_OK) return rc;
  const int chunks = pairs > 0 ? sgemm::plan_chunks(pairs) : 1;
  const sgemm::PlanArgs p{(int)pairs, (int)first, (int)groups, sgemm::plan_chunk(pairs), chunks,
                          picks, offsets, sources, places, static_cast<int *>(workspace)};
  return status(sgemm::launch_route_plan(p, stream_of(stream)));
}

int sgemm_rows_gather(int64_t rows, int64_t pairs, int64_t topk, int64_t N, int type,
                      const void *X, int64_t ldx, const int32_t *sources, const float *weights,
                      void *Y, int64_t ldy, void *stream) {
  const int64_t wide = N > 1 ? N : 1;
  if (rows < 0 || pairs < 0 || topk < 1 || N < 0 || bad_type(type) || pairs % topk != 0 ||
      ldx < wide || ldy < wide)
    return SGEMM_ERR_INVALID_VALUE;
  int rc = check_rows(rows, rows, N, type, ldx, ldy);
  if (rc != SGEMM_OK) return rc;
  if (pairs > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  const bool writes = rows > 0 && N > 0 && pairs > 0;
  if (writes && (bad_pointer(X, size_of(type)) || bad_pointer(Y, size_of(type)) ||
                 bad_pointer(sources, 4) || misaligned(weights, 4)))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  if ((rc = launchable()) != SGEMM_OK) return rc;
  const sgemm::RowsArgs p{(int)rows, (int)topk, (int)N, (int)pairs, X, ldx, sources, weights, Y,
                          ldy, sgemm::make_fast_div(pieces_of(N, type)), pieces_of(N, type)};
  return status(sgemm::launch_rows_gather(p, type == SGEMM_TYPE_BF16, stream_of(stream)));
}

int sgemm_rows_combine(int64_t tokens, int64_t topk, int64_t rows, int64_t N, int type,
                       const void *X, int64_t ldx, const int32_t *places, const float *weights,
                       void *Y, int64_t ldy, void *stream) {
  const int64_t wide = N > 1 ? N : 1;
  if (tokens < 0 || topk < 1 || rows < 0 || N < 0 || bad_type(type) || ldx < wide || ldy < wide)
    return SGEMM_ERR_INVALID_VALUE;
  int rc = check_rows(tokens, tokens, N, type, ldx, ldy);
  if (rc != SGEMM_OK) return rc;
  if (rows > kMaxDim || (tokens > 0 && topk > kMaxDim / tokens)) return SGEMM_ERR_TOO_LARGE;
  const bool writes = tokens > 0 && N > 0;
  if (writes && (bad_pointer(Y, size_of(type)) || bad_pointer(places, 4) ||
                 misaligned(weights, 4) || (rows > 0 && bad_pointer(X, size_of(type)))))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  if ((rc = launchable()) != SGEMM_OK) return rc;
  const sgemm::RowsArgs p{(int)tokens, (int)topk, (int)N, (int)rows, X, ldx, places, weights, Y,
                          ldy, sgemm::make_fast_div(pieces_of(N, type)), pieces_of(N, type)};
  return status(sgemm::launch_rows_combine(p, type == SGEMM_TYPE_BF16, stream_of(stream)));
}

int sgemm_rows_combine_backward(int64_t tokens, int64_t topk, int64_t rows, int64_t N, int type,
                                const void *X, int64_t ldx, const void *dY, int64_t lddy,
                                const int32_t *places, const float *weights, void *dX,
                                int64_t lddx, float *dweights, void *stream) {
  const int64_t wide = N > 1 ? N : 1;
  if (tokens < 0 || topk < 1 || rows < 0 || N < 0 || bad_type(type) || lddy < wide ||
      (dweights && ldx < wide) || (dX && lddx < wide))
    return SGEMM_ERR_INVALID_VALUE;
  if (tokens > 0 && topk > kMaxDim / tokens) return SGEMM_ERR_TOO_LARGE;
  int rc = check_rows(rows, tokens * topk, N, type, dweights ? ldx : 1, lddy);
  if (rc != SGEMM_OK) return rc;
  if (dX && lddx > kMaxDim) return SGEMM_ERR_TOO_LARGE;
  const bool writes = tokens > 0 && (dweights || (dX && N > 0));
  const unsigned size = size_of(type);
  if (writes && (bad_pointer(places, 4) || misaligned(weights, 4) || misaligned(dX, size) ||
                 misaligned(dweights, 4) || (N > 0 && bad_pointer(dY, size)) ||
                 (dweights && rows > 0 && N > 0 && bad_pointer(X, size))))
    return SGEMM_ERR_INVALID_VALUE;
  if (!sgemm_api::ready()) return SGEMM_ERR_NOT_INITIALIZED;
  if (!writes) return SGEMM_OK;
  if ((rc = launchable()) != SGEMM_OK) return rc;
  const sgemm::RowsBackArgs p{(int)(tokens * topk), (int)topk, (int)N, (int)rows, X, ldx, dY,
                              lddy, places, weights, dX, lddx, dweights};
  return status(sgemm::launch_rows_combine_backward(p, type == SGEMM_TYPE_BF16, stream_of(stream)));
}

}  // extern "C"
