/*
 * mmac, 4-bit block-scaled operands: packed FP4_E2M1 elements with one E8M0 scale
 * per 32 consecutive elements of a row.  Part of libmmac.so; the conventions of mmac.h
 * (layouts, alignment, memory, asynchrony, errors, thread safety) hold here too; an
 * operand without elements may be NULL and of any pitch.
 */
#ifndef MMAC_MX4_H
#define MMAC_MX4_H

#include "mmac_lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows to 4 bits: X (x_type F16, BF16 or F32, row-major M x K, 16-byte alignment
 * and pitch) -> the packed FP4_E2M1 elements and scale words that mmac_gemm_dense_mx and
 * mmac_gemm_grouped_mx read (rows of 16*ceil(K/32) bytes, `pitch` bytes apart, a
 * multiple of 16; SX as in mmac_lowbit.h).  Exponents as in mmac_mx8_quantize with T = 6;
 * each element is the E2M1 value nearest to x * 2^(127-e), ties to the even code, with
 * x's sign.  Nothing saturates.  A block that holds a NaN or an infinity gets e = 255
 * and zero codes, which is NaN to both products.  Codes past K are zero.
 */
mmac_status_t mmac_mx4_quantize(mmac_dtype_t x_type, int64_t M, int64_t K, const void *X, int64_t ldx, void *Xq,
                                int64_t pitch, uint32_t *SX, int64_t lds, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MMAC_MX4_H */
