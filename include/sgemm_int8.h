/*
 * sgemm_int8.h -- matrices held in 8-bit integers with a scale for each row, and
 * their products on the integer matrix cores of MI355X (gfx950); part of
 * libsgemm.so.
 *
 * The format.  A row of K values (a token's activations, or the weights of an
 * output channel) is held as codes -127 .. 127 and one single-precision scale;
 * an element is their product.
 *
 * The cast.  scale = (the row's largest magnitude) / 127, rounded to single
 * precision; code = the whole number nearest to value / scale, halves to the
 * even one (the quotient itself is not rounded first), at most 127 in magnitude
 * (a bound that is met only where the scale is subnormal).  Where the scale is 0
 * the codes are 0.  A row with a NaN or an infinity gets scale NaN and codes 0: every
 * product with it is NaN.
 *
 * How a matrix of `rows` x K is held.  codes: rows of ldq bytes, of which the
 * first Kp, K padded to the next multiple of 128, are used; those from K on are
 * zeros (the products below require that of at least one operand).  ldq >= Kp, a
 * multiple of 16; the codes' address is a multiple of 16.  scales: `rows`
 * floats, 4-byte aligned.  Any consecutive rows of a held matrix are a held
 * matrix too.  Codes of -128 are allowed in products.
 *
 * Limits (SGEMM_ERR_TOO_LARGE): sizes and leading dimensions below 2^31, K <
 * 2^17 (a sum of K products of codes fits 32 bits), ldq of a product's operands
 * below 2^22, ldc of the products below 2^27, each launch below 2^32 work-items.
 * Everything else -- ownership, streams, asynchrony, no allocation, status
 * codes, checks of arguments before the runtime -- is as in sgemm.h.
 */
#ifndef SGEMM_INT8_H_
#define SGEMM_INT8_H_

#include <stdint.h>

#include "sgemm.h"
#include "sgemm_mxfp4.h" /* SGEMM_TYPE_F32, SGEMM_TYPE_BF16 */

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of operands that are held as above. */
#define SGEMM_TYPE_INT8 3

/* Bytes of the codes of a held matrix with ldq = Kp, or a negative status. */
int64_t sgemm_int8_codes_size(int64_t rows, int64_t K);

/*
 * Cast to the format.  X holds single-precision or bfloat16 values (`type`),
 * rows x K with leading dimension ldx >= max(1, K), or with trans == 1 the
 * transpose, K x rows with ldx >= max(1, rows) -- how sgemm_run takes a B
 * whose columns are output channels.  Writes the Kp bytes of each row of the
 * codes, padding included, and the scales.  rows == 0 or K == 0 is a no-op.
 */
int sgemm_int8_quantize(int trans, int64_t rows, int64_t K, int type, const void *X, int64_t ldx,
                        void *codes, int64_t ldq, float *scales, void *stream);

/*
 * C = alpha * A B^T + beta * C, where B is a held matrix of N rows by K and A is
 * M x K:
 *   typeA == SGEMM_TYPE_INT8            held: A points to its codes, lda is
 *                                       their ldq, scalesA the scales;
 *   SGEMM_TYPE_F32, SGEMM_TYPE_BF16     values with leading dimension lda >=
 *                                       max(1, K), cast on the way; scalesA is
 *                                       not used.
 * Casting on the way gives the bits of sgemm_int8_quantize followed by the
 * product of held matrices.  C is M x N of typeC (SGEMM_TYPE_F32 or
 * SGEMM_TYPE_BF16), ldc >= max(1, N).  The sum of the codes' products is exact;
 *   v = ((float)sum * scaleA(m)) * scaleB(n),
 *   C = alpha v, or fma(alpha, v, beta C),
 * each step rounded to single precision and a bfloat16 C once more, to the
 * nearest, ties to even.  So before that last rounding, while nothing leaves the
 * normal range, |C - exact| <= 5 2^-24 (|alpha v| + |beta C|), and results are
 * the same bits whatever the sizes around them.  C is not read when beta == 0;
 * A and B are not read when alpha == 0 or K == 0.
 *
 * Workspace: device memory of at least sgemm_int8_workspace_size(typeA, M, K)
 * bytes (0 for SGEMM_TYPE_INT8), 16-byte aligned, in which a call keeps the
 * cast A.  Its contents have no meaning between calls; two calls that may run
 * at the same time, two captured graphs among them, must not share one.
 * SGEMM_ERR_INVALID_VALUE for a null, misaligned or too small workspace where
 * one is needed (M, N, K positive, alpha != 0, A not held).
 */
int64_t sgemm_int8_workspace_size(int typeA, int64_t M, int64_t K);

int sgemm_run_int8(int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
                   int64_t lda, const float *scalesA, const void *B, int64_t ldb,
                   const float *scalesB, float beta, int typeC, void *C, int64_t ldc,
                   void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The same, grouped: for every group g and each of its rows r,
 *   C(r, :) = alpha * A(r, :) B_g^T + beta * C(r, :)
 * where B is a held matrix of groups * N rows and B_g its rows g * N to
 * g * N + N - 1.  `offsets` and `groups` are as in sgemm_grouped.h; rows that
 * belong to no group are not written, and what A holds there affects nothing.
 */
int sgemm_run_int8_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                           int typeA, const void *A, int64_t lda, const float *scalesA,
                           const void *B, int64_t ldb, const float *scalesB, float beta,
                           int typeC, void *C, int64_t ldc, const int64_t *offsets,
                           void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_INT8_H_ */
