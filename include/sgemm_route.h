/*
 * sgemm_route.h -- routing of rows (tokens) to experts, and taking rows to their
 * experts and back, on MI355X (gfx950); part of libsgemm.so.
 *
 * A layer of experts runs
 *   sgemm_route                 which experts each token goes to, with weights
 *   sgemm_route_plan            the pairs (token, pick) sorted by expert: the
 *                               offsets that sgemm_run_grouped, sgemm_run_grouped_k,
 *                               sgemm_run_int8_grouped and sgemm_run_mxfp4_grouped
 *                               read, and where each row comes from and goes to
 *   sgemm_rows_gather           the tokens' rows in that order
 *   (the products, grouped)
 *   sgemm_rows_combine          the experts' rows back to tokens, weighted and added
 * and backwards sgemm_rows_combine_backward, the products' gradients,
 * sgemm_rows_combine without weights (the gradient of sgemm_rows_gather without
 * them) and sgemm_route_backward.  Nothing is read on the host: the calls can be captured
 * into a graph that is replayed with other tokens.
 *
 * Element types are SGEMM_TYPE_F32 and SGEMM_TYPE_BF16 (`type`), of every matrix
 * of a call but the weights, which are single precision.  Ownership, streams,
 * asynchrony, no allocation, status codes and checks of arguments before the
 * runtime are as in sgemm.h; pointers must be aligned to their elements
 * (SGEMM_ERR_INVALID_VALUE), offsets to 8 bytes.  Outputs must not overlap inputs.
 * Limits (SGEMM_ERR_TOO_LARGE): sizes and leading dimensions below 2^31, pairs =
 * tokens * topk too, each launch below 2^32 work-items (a wave of 64 for each
 * token in sgemm_route and sgemm_route_backward; for each row that is written and
 * 4096 bytes of it in sgemm_rows_gather and sgemm_rows_combine, for each pair and
 * 4096 bytes in sgemm_rows_combine_backward).
 */
#ifndef SGEMM_ROUTE_H_
#define SGEMM_ROUTE_H_

#include <stdint.h>

#include "sgemm.h"
#include "sgemm_mxfp4.h" /* SGEMM_TYPE_F32, SGEMM_TYPE_BF16 */

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_ROUTE_MAX_EXPERTS 1024
#define SGEMM_ROUTE_MAX_TOPK 64
#define SGEMM_ROUTE_MAX_GROUPS 64

/* How scores are made of logits. */
#define SGEMM_SCORE_SOFTMAX 0
#define SGEMM_SCORE_SIGMOID 1

/*
 * For each token t, with l the logits at t * ldl (ldl >= experts):
 *   s = softmax(l) over the experts, or sigmoid(l)
 *   c = s + bias              (bias: `experts` floats, or null for none)
 * The experts lie in `groups` groups of experts / groups consecutive ones (1: no
 * groups).  A group's score is the sum of its group_top (1 or 2) highest c.
 * The topk_groups groups with the highest scores are kept, and among their
 * experts the topk with the highest c are picked.  Equal ones: the lowest
 * index.  Then, over j < topk,
 *   picks[t * topk + j]   = the expert, in falling order of c
 *   weights[t * topk + j] = scale * s(pick), or, with renormalize == 1,
 *                           scale * s(pick) / (sum of the picked s).
 * Comparisons are those of the formulas in double precision, so that picks do
 * not depend on how an exponential is rounded to single precision; without bias
 * and groups they are those of the logits.  Weights are single precision, off by
 * a few roundings.
 *
 * A logit or a bias of -infinity disables an expert: it is never picked, and
 * counts for nothing in its group's score (a group with no other expert comes
 * last).  Where fewer than topk experts can be picked, the last picks are -1
 * with weight 0; without any all are.  Picked scores that sum to 0 (by
 * underflow) renormalise to 0.  A row with a NaN, and under softmax one with a
 * +infinity, gets NaN weights; its picks are some distinct experts or -1, as are
 * those of all rows where a bias is NaN.
 *
 * 1 <= topk <= min(experts, SGEMM_ROUTE_MAX_TOPK), 1 <= experts, groups a divisor
 * of experts, 1 <= topk_groups <= groups, group_top 1 or 2
 * (SGEMM_ERR_INVALID_VALUE); experts <= SGEMM_ROUTE_MAX_EXPERTS, groups <=
 * SGEMM_ROUTE_MAX_GROUPS (SGEMM_ERR_TOO_LARGE).  tokens == 0 is a no-op.
 */
int sgemm_route(int64_t tokens, int64_t experts, int64_t topk, int score, int type,
                const void *logits, int64_t ldl, const float *bias, int64_t groups,
                int64_t topk_groups, int64_t group_top, int renormalize, float scale,
                int32_t *picks, float *weights, void *stream);

/*
 * The gradient of the weights with respect to the logits, the picks held: for
 * dweights (tokens x topk) writes dlogits (tokens x experts, ldd >= experts), of
 * the logits' type, computed in single precision and rounded once.  Experts
 * that were not picked get 0, except under softmax without renormalize.  Picks
 * that are not in [0, experts) are left out, as are those of disabled experts;
 * an expert must not be among a token's picks twice.
 */
int sgemm_route_backward(int64_t tokens, int64_t experts, int64_t topk, int score, int type,
                         const void *logits, int64_t ldl, int renormalize, float scale,
                         const int32_t *picks, const float *dweights, void *dlogits, int64_t ldd,
                         void *stream);

/*
 * Sort pairs by expert.  Pair p (token p / topk, its pick p % topk) goes to
 * group picks[p] - first if that lies in [0, groups); others go to no group (a
 * device that holds experts first .. first + groups - 1 leaves out the rest).
 * Writes
 *   offsets[g], g <= groups   the rows of group g are offsets[g] .. offsets[g + 1] - 1
 *   sources[r], r < pairs     the pair of row r, -1 from offsets[groups] on
 *   places[p], p < pairs      the row of pair p, -1 where it has none.
 * Inside a group pairs keep their order.  groups <= 4096 (SGEMM_ERR_TOO_LARGE),
 * first >= 0.  groups == 0 or pairs == 0: all offsets are 0.
 *
 * Workspace: device memory of sgemm_route_plan_workspace_size(pairs, groups)
 * bytes, 16-byte aligned; nothing in it has a meaning between calls, and two
 * calls that may run at the same time, two captured graphs among them, must not
 * share one.
 */
int64_t sgemm_route_plan_workspace_size(int64_t pairs, int64_t groups);

int sgemm_route_plan(int64_t pairs, int64_t first, int64_t groups, const int32_t *picks,
                     int64_t *offsets, int32_t *sources, int32_t *places, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * Y(r, :) = w(sources[r]) * X(sources[r] / topk, :) for r < rows, over N columns;
 * w = weights[pair], or 1 where weights is null (a copy of the bits).  Rows
 * whose source is not in [0, pairs) are not written; X has pairs / topk rows
 * (pairs a multiple of topk).  One rounding, of the product.
 *
 * Its gradients, for dY that of Y and the plan's places: of X, sgemm_rows_combine of dY
 * with the same weights; of the weights, sgemm_rows_combine_backward with dY in
 * the place of its X and X in that of its dY, weights and dX null.
 */
int sgemm_rows_gather(int64_t rows, int64_t pairs, int64_t topk, int64_t N, int type,
                      const void *X, int64_t ldx, const int32_t *sources, const float *weights,
                      void *Y, int64_t ldy, void *stream);

/*
 * Y(t, :) = sum_j w(t, j) * X(places[t * topk + j], :) for t < tokens, over N
 * columns; w = weights[t * topk + j], or 1 where weights is null.  X has `rows`
 * rows; places not in [0, rows) add nothing, whatever the weight.  Sums are single
 * precision in the order of j (fused multiply-adds), rounded once to the type.  A
 * token without a place gets zeros.
 */
int sgemm_rows_combine(int64_t tokens, int64_t topk, int64_t rows, int64_t N, int type,
                       const void *X, int64_t ldx, const int32_t *places, const float *weights,
                       void *Y, int64_t ldy, void *stream);

/*
 * The gradients of sgemm_rows_combine.  For every pair p = t * topk + j with
 * places[p] in [0, rows):
 *   dX(places[p], :) = weights[p] * dY(t, :)       (weights null: 1)
 *   dweights[p]      = sum_n X(places[p], n) * dY(t, n)
 * dweights of other pairs is 0, and rows of dX that no pair has are not written.
 * dX or dweights may be null and is left out then; X is read only for dweights.
 * Sums are single precision in an order that is fixed for N.  No two pairs may
 * have the same place.
 */
int sgemm_rows_combine_backward(int64_t tokens, int64_t topk, int64_t rows, int64_t N, int type,
                                const void *X, int64_t ldx, const void *dY, int64_t lddy,
                                const int32_t *places, const float *weights, void *dX,
                                int64_t lddx, float *dweights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_ROUTE_H_ */
