/*
 * mmac, products grouped by expert: the rows of A are sorted by group, each group
 * has a weight matrix of its own, and where the groups begin is known in GPU
 * memory only.  Part of libmmac.so; the conventions of mmac.h (layouts, alignment,
 * memory, asynchrony, errors, thread safety, alpha and beta) hold here too; an
 * operand without elements may be NULL and of any pitch.
 *
 *   groups   their number G, at most 2^30 (MMAC_ERR_UNSUPPORTED beyond).
 *   offsets  G + 1 32-bit integers in device memory, not decreasing, from 0 to M:
 *            rows offsets[g] .. offsets[g+1] - 1 belong to group g, which may have none.
 *            Rows before offsets[0] and from offsets[G] on belong to no group: they are
 *            not read, and those of D stay as they were.  (Offsets that break these rules
 *            give unspecified values in D; nothing outside the arrays is touched.)
 *   B        group g's matrix is at B + g * stride_b elements; all have one shape
 *            and pitch.  stride_b * element size must be a multiple of 16 bytes and
 *            at least the matrix's own extent (one group: anything).
 * The tile a product runs in is picked on the host from M / G, the rows of an
 * average group; MMAC_TILE (256, 1282 for 128 x 256, 128, 64; forward products of
 * K-contiguous weights also 32 and 16) overrides it.
 */
#ifndef MMAC_GROUPED_H
#define MMAC_GROUPED_H

#include "mmac_lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * For every group g and its rows i:
 *   D[i] = round(act(alpha * A[i] * B_g + beta * C[i] + bias_g))
 *   a_type    F16 or BF16, A and B alike.
 *   trans_b   0: B_g is column-major K x N (N rows of K elements, ldb >= K), as in
 *             mmac_gemm_dense: the forward product of N x K weights.  1: it is row-major
 *             K x N (K rows of N elements, ldb >= N, K * ldb * 2 below 2^31 bytes): with the
 *             same weights, their N as this K, the gradient of the forward product's input.
 *   A, C, D   M rows; ep as in mmac_gemm_dense_ep, but ep->bias holds G rows of N values.
 * M, N or G == 0: nothing is done.  K == 0: the sum is zero (A and B are not read).  More than
 * 4 million tiles of 256 x 256 (128 x 256 in mmac_gemm_grouped_mx), each group's counted
 * up to whole ones in the worst spread of the rows: MMAC_ERR_UNSUPPORTED.
 */
mmac_status_t mmac_gemm_grouped(mmac_dtype_t a_type, int trans_b, int64_t groups, int64_t M, int64_t N, int64_t K,
                                double alpha, const void *A, int64_t lda, const int32_t *offsets, const void *B,
                                int64_t ldb, int64_t stride_b, double beta, const void *C, int64_t ldc, void *D,
                                int64_t ldd, const mmac_epilogue_t *ep, void *stream);

/*
 * The forward product from block-scaled operands: A an mx8 matrix (Xq, SX of
 * mmac_lowbit.h: a_type FP8_E4M3 or BF8_E5M2), B_g the B of mmac_gemm_dense_mx, 8-bit
 * (b_type FP8_E4M3 or BF8_E5M2) or packed FP4_E2M1 (mmac_mx4_quantize).  K % 32 == 0.
 *   SA        ceil(K/128) x ldsa words, ldsa >= M, 4-byte aligned; SB group g's words
 *             are at SB + g * stride_sb, ceil(K/128) x ldsb, ldsb >= N, 4-byte aligned.
 *             Each array (a group's, for B) spans less than 2^31 bytes.
 *   lda, ldb, stride_b count elements (FP4: two per byte; rows start on 16 bytes).
 * e = 255 (NaN) in a block that is used gives NaN in the outputs whose sums hold it.
 * Sums are fp32.  Outputs of 16 and 8 bits come from the block-scaled matrix instructions,
 * for any exponents; they add up the 64 or 128 products of an instruction with fewer bits than
 * fp32, an error of up to 2^-13 of the sum of the magnitudes before the output is rounded.  Where the
 * terms cancel, that may be more than the rounding (random signs, K 8192: 1.3 % of bf16 outputs are
 * not the nearest, the normwise error against 64 bits grows by less than 1e-4 of itself).  For fp32 outputs
 * the elements times their scales become bf16, exact for magnitudes from 2^-126 to bf16's
 * largest, and their products are exact.  The rest as in mmac_gemm_grouped.
 */
mmac_status_t mmac_gemm_grouped_mx(mmac_dtype_t a_type, mmac_dtype_t b_type, int64_t groups, int64_t M, int64_t N,
                                   int64_t K, double alpha, const void *A, int64_t lda, const uint32_t *SA,
                                   int64_t ldsa, const int32_t *offsets, const void *B, int64_t ldb, int64_t stride_b,
                                   const uint32_t *SB, int64_t ldsb, int64_t stride_sb, double beta, const void *C,
                                   int64_t ldc, void *D, int64_t ldd, const mmac_epilogue_t *ep, void *stream);

/*
 * The gradient of the weights: for every group g, with the sum over its rows i,
 *   D_g = alpha * sum_i dY[i]^T * X[i] + beta * C_g        (N x K, row-major)
 *   y_type    F16 or BF16, dY (M x N) and X (M x K) alike.
 *   D, C      group g's matrix is at D + g * stride_d (C + g * stride_c) elements;
 *             stride_d >= (N - 1) * ldd + K.
 *   ep        NULL, or d_type with act NONE and bias NULL (MMAC_ERR_UNSUPPORTED otherwise).
 * A group without rows: D_g = beta * C_g.  Rows of no group do not count.  More than 4 million
 * tiles of 256 x 256 (each group's counted up to whole ones): MMAC_ERR_UNSUPPORTED.
 */
mmac_status_t mmac_gemm_grouped_wgrad(mmac_dtype_t y_type, int64_t groups, int64_t M, int64_t N, int64_t K,
                                      double alpha, const void *dY, int64_t ldy, const void *X, int64_t ldx,
                                      const int32_t *offsets, double beta, const void *C, int64_t ldc,
                                      int64_t stride_c, void *D, int64_t ldd, int64_t stride_d,
                                      const mmac_epilogue_t *ep, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MMAC_GROUPED_H */
