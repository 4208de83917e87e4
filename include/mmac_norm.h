/*
 * mmac, the root-mean-square norm in front of a product: the addition of the
 * residual stream, the norm, and its output in 16 bits, 32 bits or as the 8-bit
 * block-scaled operand (an "mx8" matrix of mmac_lowbit.h) that
 * mmac_gemm_dense_mx, mmac_gemm_grouped_mx and mmac_gemm_mx8_wgrad read; and its
 * gradients.  Part of libmmac.so; the conventions of mmac.h (alignment, memory,
 * asynchrony, errors, thread safety) hold here too; an operand without elements
 * may be NULL and of any pitch.  Every matrix is row-major M x N with 16-byte alignment and pitch,
 * ld in elements; N is the length that is normed, M the number of rows.
 */
#ifndef MMAC_NORM_H
#define MMAC_NORM_H

#include "mmac_lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Per row:
 *   h = X                              (residual == NULL)
 *   h = round(X + residual)            (rounded to x_type as the epilogues of mmac.h round)
 *   r = 1 / sqrt(mean(h^2) + eps)
 *   y = h * r * w
 * Sums, r and y are fp32; the norm is that of h as it is kept.
 *   x_type    F16, BF16 or F32: X, residual and H.
 *   w_type    x_type or F32: w, N values, 16-byte aligned.
 *   y_type    x_type: Y is the matrix y, rounded like h (ldy >= N; SY and lds unused).
 *             FP8_E4M3 or BF8_E5M2: Y and SY are the mx8 matrix that mmac_mx8_quantize
 *             makes of y in fp32 (ldy >= 32*ceil(N/32), lds >= M).
 *   residual  NULL (ldr unused) or the stream that X is added to.
 *   H         NULL (ldh unused) or where h goes.
 *   rstd      NULL or M fp32 values, where r goes.
 *   eps       finite, not negative.  With eps = 0 a row of zeros gives NaN.
 * H may be X or residual, and Y may be X when it has x_type, with the same
 * pitch (but H, Y and the other input are then apart); other overlaps are not allowed.
 * M == 0 or N == 0: nothing is done.  A row with a NaN or an infinity, or whose
 * sum of squares passes fp32, is what the formulas give in fp32.
 */
mmac_status_t mmac_rmsnorm(mmac_dtype_t x_type, mmac_dtype_t w_type, mmac_dtype_t y_type, int64_t M, int64_t N,
                           const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *w, double eps,
                           void *H, int64_t ldh, void *Y, int64_t ldy, uint32_t *SY, int64_t lds, float *rstd,
                           void *stream);

/*
 * The gradients, given dY, that of y, and the forward pass's h and r:
 *   v  = w * dY,  x = h * r
 *   dX = r * (v - x * mean(v * x)) + dH          (that of X and of the residual alike)
 *   dW = the sum over the rows of dY * x         (fp32)
 *   x_type    F16, BF16 or F32: dY, H, dH and dX.  w_type as above.
 *   dH        NULL (lddh unused) or the gradient that reaches h on the residual stream.
 *   dW        NULL, or N fp32 values, 16-byte aligned.
 *   workspace device memory, 16-byte aligned, for the partial sums of dW: at least
 *             mmac_rmsnorm_grad_workspace_bytes (MMAC_ERR_INVALID_ARG otherwise); unused
 *             without dW.  It need not be cleared, and its first KiB is left alone, so
 *             it may be a workspace that the products share, in one stream.
 * dX may be dY or dH (with the same pitch).  The sums are added up in a fixed order:
 * the results do not depend on timing.  M == 0: dW is zero, and only that is done.  N == 0: nothing is done.
 */
mmac_status_t mmac_rmsnorm_grad(mmac_dtype_t x_type, mmac_dtype_t w_type, int64_t M, int64_t N, const void *dY,
                                int64_t lddy, const void *H, int64_t ldh, const void *w, const float *rstd,
                                const void *dH, int64_t lddh, void *dX, int64_t lddx, float *dW, void *workspace,
                                int64_t workspace_bytes, void *stream);

/* Workspace bytes of mmac_rmsnorm_grad with a dW.  Host-only. */
int64_t mmac_rmsnorm_grad_workspace_bytes(int64_t M, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* MMAC_NORM_H */
