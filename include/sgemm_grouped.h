/*
 * sgemm_grouped.h -- single-precision products whose rows fall into groups of
 * unequal length, each group with a matrix of its own, on MI355X (gfx950);
 * part of libsgemm.so.
 *
 * A layer of experts sorts its rows (tokens) by the expert that a router
 * picked for them; how many each expert gets is known on the device only.
 * The group lengths are therefore read from device memory by the kernels:
 * the calls need no copy to the host and can be captured into a graph that
 * is replayed with other lengths.
 *
 * Groups.  `offsets` is a device array of groups + 1 values: group g has the
 * rows offsets[g] <= r < offsets[g + 1].  They must not decrease and must lie
 * in [0, rows], where `rows` is M of sgemm_run_grouped and K of
 * sgemm_run_grouped_k.  Rows before offsets[0] and from offsets[groups] on
 * belong to no group: they are neither read nor written.  A group may be
 * empty.  The host cannot check these values.  A kernel clamps each group's
 * range to [0, rows] (and to length zero where it decreases), so nothing
 * outside the operands is read or written whatever they are; where groups
 * overlap, which of them C holds in the rows they share is undefined, and
 * some rows may be left out.
 *
 * Layout, numerics, streams, pointers, status codes and the order of checks
 * are those of sgemm.h: row-major single precision, the accuracy contract
 * |C(i,j) - exact| <= 1e-5 * sum |products| + 1e-6 for the sum, the order
 * of summation fixed for a given call and group lengths (repeated calls give
 * identical bits), results rounded once after beta * C, C not read when
 * beta == 0, A and B not read when alpha == 0.  The contract holds whatever
 * the products' signs, for sums over up to 2^29 (long sums are added up in
 * parts, so that their roundings do not pile up).  Any 4-byte alignment of A, B
 * and C is accepted; offsets must be 8-byte aligned
 * (SGEMM_ERR_INVALID_VALUE).  The calls allocate nothing, use no workspace
 * and are asynchronous on `stream`.  Limits (SGEMM_ERR_TOO_LARGE): sizes
 * below 2^31, groups <= SGEMM_GROUPED_MAX_GROUPS, one launch below 2^32
 * work-items at 256 for each 32 x 32 block of C (sgemm_run_grouped counts
 * one partly filled row of blocks for each group), lda and ldb below 2^22
 * where A and B are read, ldc below 2^27, and K of sgemm_run_grouped_k at
 * most 2^30.
 */
#ifndef SGEMM_GROUPED_H_
#define SGEMM_GROUPED_H_

#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_GROUPED_MAX_GROUPS 4096

/*
 * For every group g and each of its rows r:
 *   C(r, :) = alpha * A(r, :) op(B_g) + beta * C(r, :)
 * A is M x K (lda >= max(1, K)), C is M x N (ldc >= max(1, N)).  B_g starts
 * g * strideB floats after B: K x N (transB == 0, ldb >= max(1, N)) or the
 * transpose of a stored N x K matrix (transB == 1, ldb >= max(1, K));
 * strideB >= 0, and 0 shares one matrix between the groups.  With B_g the
 * weights of expert g this is a layer's forward product; with the other
 * value of transB and the output's gradient as A it gives the gradient of
 * the layer's input.  M == 0, N == 0 or groups == 0 is a no-op; K == 0 or
 * alpha == 0 leaves beta * C in the groups' rows.
 */
int sgemm_run_grouped(int transB, int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                      const float *A, int64_t lda, const float *B, int64_t ldb, int64_t strideB,
                      float beta, float *C, int64_t ldc, const int64_t *offsets, void *stream);

/*
 * For every group g, over its rows r:
 *   C_g = alpha * sum_r A(r, :)^T B(r, :) + beta * C_g
 * A is K x M (lda >= max(1, M)), B is K x N (ldb >= max(1, N)); C_g is M x N
 * (ldc >= max(1, N)) and starts g * strideC floats after C (strideC >= 0),
 * the matrices of different groups disjoint (groups > 1: strideC >=
 * (M - 1) * ldc + N).
 * With A a layer's input and B its output's gradient this is the gradient of
 * each expert's weights.  An empty group leaves beta * C_g (zeros when
 * beta == 0).  M == 0, N == 0 or groups == 0 is a no-op.
 */
int sgemm_run_grouped_k(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                        const float *A, int64_t lda, const float *B, int64_t ldb, float beta,
                        float *C, int64_t ldc, int64_t strideC, const int64_t *offsets,
                        void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GROUPED_H_ */
