/*
 * sgemm_orthogonalize.h -- matrices brought towards orthogonal ones by Newton-Schulz
 * products, on MI355X (gfx950); part of libsgemm.so.
 *
 * An optimiser replaces the update X of a weight matrix (its momentum) by the
 * nearest matrix with orthonormal rows or columns, or near enough: with the
 * singular value decomposition X = U diag(s) V^T, by U diag(f(s)) V^T with f(s)
 * around 1.  The update of every expert's weights, as sgemm_run_grouped_k
 * accumulates their gradients, is a batch of such matrices.
 *
 * The operation.  For each matrix of the batch, with |X| the root of the sum of
 * its squares,
 *   Z = X / (|X| + eps), transposed where M > N, so that Z is m x n with m <= n
 *   `steps` times, with the step's a, b, c:   S = Z Z^T,   Z = a Z + (b S + c S S) Z
 *   Y = alpha Z, transposed back.
 * A singular value s of Z becomes a s + b s^3 + c s^5 in each step.  A matrix of
 * zeros gives zeros.
 *
 * Numerics.  Norms are summed in double precision.  The products run on the
 * half-precision matrix cores: each operand, Z between the steps among them, is
 * held as the sum of two half-precision numbers, 22 bits, under a power of two
 * for each row, and three of the four products of the pieces are added up in
 * single precision.  A product of operands is off by 3 2^-22 of itself at most,
 * where one in single precision is off by 2^-24; sums of many differ by less.
 * A row's power of two goes by the row's own norm as it was up to eight steps
 * before, times what the polynomials can have made of it since (and at most by the
 * largest singular value there can be): an element is off by 2^-40 of that range
 * at most, of its row's range and of its column's, so that rows or columns that
 * are small against the others keep their digits.  What is in a small row and a
 * small column, far below either's range, keeps them while the product of the steps'
 * largest |a + b s^2 + c s^4| stays below about 2^15 (eight steps of 3.44): past
 * that such a column (of M x N with M > N, such a row) loses digits, and the others
 * do not.  Where one side is longer than about the square of the other, runs of
 * its rows or columns share a range, the largest of theirs.
 * Matrices with M <= 64 or N <= 64 are multiplied in single precision instead.  Sums
 * are taken in an order that is fixed for a matrix' sizes, so repeated calls give
 * identical bits, whatever the batch around a matrix.  X has to be finite.
 *
 * Ranges.  `coefficients` are on the host, read during the call: 3 * sets floats,
 * a, b, c of each step, with sets == steps, or sets == 1 for all steps alike.
 * They have to be finite, and the polynomials must not take a singular value that
 * starts at 1 or below past 2^16 (SGEMM_ERR_INVALID_VALUE).  1 <= steps <= 64,
 * eps >= 0, alpha finite.  Element types are SGEMM_TYPE_F32 and SGEMM_TYPE_BF16;
 * a bfloat16 Y is rounded once more, to the nearest, ties to even.
 *
 * Layout.  X and Y are M x N, rows ldx (ldy) >= max(1, N) elements apart,
 * matrices strideX (strideY) apart; strideY >= (M - 1) * ldy + N where batch >
 * 1, strideX >= 0.  Y may be X (the same address, type, ld and stride); else they
 * must not overlap.  Limits (SGEMM_ERR_TOO_LARGE): M, N <= 2^20, leading
 * dimensions below 2^31, each launch below 2^32 work-items.
 *
 * Workspace: device memory of sgemm_orthogonalize_workspace_size(batch, M, N)
 * bytes, 16-byte aligned.  Its contents have no meaning between calls; two calls
 * that may run at the same time, two captured graphs among them, must not share
 * one.  Ownership, streams, asynchrony, no allocation, status codes and checks
 * of arguments before the runtime are as in sgemm.h.  batch == 0, M == 0 or N ==
 * 0 is a no-op.
 */
#ifndef SGEMM_ORTHOGONALIZE_H_
#define SGEMM_ORTHOGONALIZE_H_

#include <stdint.h>

#include "sgemm.h"
#include "sgemm_mxfp4.h" /* SGEMM_TYPE_F32, SGEMM_TYPE_BF16 */

#ifdef __cplusplus
extern "C" {
#endif

int64_t sgemm_orthogonalize_workspace_size(int64_t batch, int64_t M, int64_t N);

int sgemm_orthogonalize(int64_t batch, int64_t M, int64_t N, int64_t steps, int64_t sets,
                        const float *coefficients, float eps, float alpha, int typeX,
                        const void *X, int64_t ldx, int64_t strideX, int typeY, void *Y,
                        int64_t ldy, int64_t strideY, void *workspace, int64_t workspace_bytes,
                        void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_ORTHOGONALIZE_H_ */
