/*
 * sgemm_mxfp4.h -- matrices held in microscaled 4-bit floating point, and
 * their products on the 4-bit matrix cores of MI355X (gfx950); part of
 * libsgemm.so.
 *
 * The format (Open Compute Project, "OCP Microscaling Formats (MX)
 * Specification", version 1.0, MXFP4).  A row's values are taken in blocks of
 * 32 consecutive k.  A block has one scale byte s, which stands for
 * 2^(s - 127) (255: NaN), and 32 codes of 4 bits, which stand for +-{0, 0.5,
 * 1, 1.5, 2, 3, 4, 6} (bit 3 the sign, bits 2:0 the index).  An element is
 * the product of the two.
 *
 * The cast.  s = max(E - 2, 0) where E is the biased exponent of the block's
 * largest magnitude (the largest power of two not above it, over the format's
 * largest power of two, 4); the code is the nearest value to element / scale,
 * ties to the even code, and 6 for anything above 6.  A block with a NaN or
 * an infinity gets s = 255 and codes 0: all 32 of its elements read as NaN.
 *
 * How a matrix of `rows` x K is held.  K is padded to Kp, the next multiple of
 * 128, with zeros.
 *   codes   [rows][Kp / 2] bytes, the even k in a byte's low half;
 *   scales  [Kp / 128][lds][4] bytes, lds >= rows: entry (g, r, b) scales
 *           elements 128 g + 32 b .. + 31 of row r.  Scales of neighbouring
 *           rows adjoin, so the matrix cores' operand loads of 32 rows by 128
 *           k read one 128-byte line of them.  Blocks past K have codes 0 and
 *           s = 0; entries of rows >= `rows` are neither read nor written.
 * codes must be 16-byte aligned and scales 4-byte aligned
 * (SGEMM_ERR_INVALID_VALUE).  Any consecutive rows of a held matrix are a held
 * matrix too, with the same lds: row r starts at codes + r * Kp / 2 and
 * scales + 4 * r.  The calls below that read a held matrix require padding
 * as above (or any other codes whose scale is not 255 on one side and zeros
 * on the other).
 *
 * Limits (SGEMM_ERR_TOO_LARGE): sizes below 2^31, K <= 2^21, and for each
 * launch fewer than 2^32 work-items.  Leading dimensions below 2^31, ldc of the
 * products below 2^27.
 * Everything else -- ownership, streams, asynchrony, no allocation, status
 * codes, checks of arguments before the runtime -- is as in sgemm.h.
 */
#ifndef SGEMM_MXFP4_H_
#define SGEMM_MXFP4_H_

#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of operands. */
#define SGEMM_TYPE_F32 0
#define SGEMM_TYPE_BF16 1
#define SGEMM_TYPE_MXFP4 2

/* Bytes of the codes, and of the scales with lds = rows, of a held matrix;
 * or a negative status. */
int64_t sgemm_mxfp4_codes_size(int64_t rows, int64_t K);
int64_t sgemm_mxfp4_scales_size(int64_t rows, int64_t K);

/*
 * Cast to the format.  X holds single-precision or bfloat16 values (`type`),
 * rows x K with leading dimension ldx >= max(1, K), or with trans == 1 the
 * transpose, K x rows with ldx >= max(1, rows) -- how sgemm_run takes a B
 * whose columns are to be quantised along k.  Writes every byte of the codes
 * and every scale of the rows, padding included.
 */
int sgemm_mxfp4_quantize(int trans, int64_t rows, int64_t K, int type, const void *X, int64_t ldx,
                         void *codes, void *scales, int64_t lds, void *stream);

/*
 * The values a held matrix stands for, laid out as X above.  Both types hold
 * them exactly, but for those of 2^128 and more (s >= 253), which become
 * infinite.
 */
int sgemm_mxfp4_dequantize(int trans, int64_t rows, int64_t K, const void *codes,
                           const void *scales, int64_t lds, int type, void *X, int64_t ldx,
                           void *stream);

/*
 * C = alpha * A B^T + beta * C, where B is a held matrix of N rows by K
 * (scales with leading dimension ldsb) and A is M x K:
 *   typeA == SGEMM_TYPE_MXFP4           held: A points to its codes, scalesA to
 *                                       its scales, lda is their lds;
 *   SGEMM_TYPE_F32, SGEMM_TYPE_BF16     values with leading dimension lda >=
 *                                       max(1, K), cast on the way; scalesA is
 *                                       not used.
 * Casting on the way gives the bits of sgemm_mxfp4_quantize followed by the
 * product of held matrices.  C is M x N of typeC (SGEMM_TYPE_F32 or
 * SGEMM_TYPE_BF16), ldc >= max(1, N).  Products of elements are exact; sums
 * are single precision in an order that is fixed for a given call.  The
 * result is alpha * sum + beta * C, rounded to single precision once after
 * beta * C (a fused multiply-add) and, for bfloat16, once more, to the
 * nearest, ties to even.  Before that last rounding
 *   |C - exact| <= max(1e-5, (K / 7 + 16) 2^-24) * sum |products| + 1e-6.
 * The second term, past 1e-5 from K = 1063 on, is for operands whose blocks
 * spread widely: a matrix instruction adds 64 or 128 products at once and
 * drops those below 2^-27 of the largest addend (K / 8 of the bound).  Sums
 * of normally distributed values, with their magnitudes too, stay within 1e-5
 * up to K = 2^21.  C is not read when beta == 0; A and B are not read when
 * alpha == 0 or K == 0.
 *
 * Workspace: device memory of at least sgemm_mxfp4_workspace_size(typeA, M,
 * K) bytes (0 for SGEMM_TYPE_MXFP4), 16-byte aligned, in which a call keeps
 * the cast A.  Its contents have no meaning between calls; two calls that may
 * run at the same time, two captured graphs among them, must not share one.
 * SGEMM_ERR_INVALID_VALUE for a null, misaligned or too small workspace where
 * one is needed (M, N, K positive, alpha != 0, A not held).
 */
int64_t sgemm_mxfp4_workspace_size(int typeA, int64_t M, int64_t K);

int sgemm_run_mxfp4(int64_t M, int64_t N, int64_t K, float alpha, int typeA, const void *A,
                    int64_t lda, const void *scalesA, const void *B, const void *scalesB,
                    int64_t ldsb, float beta, int typeC, void *C, int64_t ldc, void *workspace,
                    int64_t workspace_bytes, void *stream);

/*
 * The same, grouped: for every group g and each of its rows r,
 *   C(r, :) = alpha * A(r, :) B_g^T + beta * C(r, :)
 * where B is a held matrix of groups * N rows and B_g its rows g * N to
 * g * N + N - 1 (ldsb >= groups * N).  `offsets` and `groups` are as in
 * sgemm_grouped.h; rows that belong to no group are not written, and what A
 * holds there affects nothing.
 */
int sgemm_run_mxfp4_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, float alpha,
                            int typeA, const void *A, int64_t lda, const void *scalesA,
                            const void *B, const void *scalesB, int64_t ldsb, float beta,
                            int typeC, void *C, int64_t ldc, const int64_t *offsets,
                            void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MXFP4_H_ */
