/*
 * mmac, low-bit operands of a linear layer: 4-bit weights with group scales and
 * 8-bit block-scaled activations, each with the call that makes it and the
 * products that read it.  Part of libmmac.so; the conventions of mmac.h
 * (layouts, alignment, memory, asynchrony, errors, thread safety) hold here too;
 * an operand without elements may be NULL.
 *
 * 4-bit weights (a "w4" matrix, N x K, the B of a product)
 *   codes   two per byte, element 2m of a row in the low nibble of byte m (the
 *           packing of MMAC_FP4_E2M1).  A row is ceil(K/32) units of 16 bytes;
 *           the nibbles at and past K may hold anything.  Rows start on
 *           16-byte boundaries, `pitch` bytes apart (a multiple of 16, at least
 *           16*ceil(K/32), at most 8 MiB).
 *   group   32, 64 or 128 consecutive elements of a row share one scale word;
 *           0: the whole row does.  The last group of a row may be short.
 *   words   scale words, group-major: words[g*ldw + j] is group g of row j,
 *           ldw >= N, 4-byte aligned, (groups * ldw) * 4 below 2^31 bytes.  The
 *           top 24 bits are those of an fp32 scale s >= 0 whose lowest eight
 *           significand bits are zero (16 significant bits: every fp16 and bf16
 *           scale exactly); the low byte is the zero point z.
 *   MMAC_U4         the element with code n (0 .. 15) is (n - z) * s, z in 0 .. 15.
 *   MMAC_FP4_E2M1   it is s times the E2M1 value of n; z must be 0.
 *
 * 8-bit activations (an "mx8" matrix, M x K): the A of mmac_gemm_dense_mx, that
 * is elements of one byte (FP8_E4M3, BF8_E5M2 or I8, the last only in the calls
 * below) with one E8M0 scale per 32 consecutive elements of a row.
 *   elements  row-major, rows of Kp = 32*ceil(K/32) elements, ld >= Kp,
 *           ld % 16 == 0, 16-byte aligned; those at and past K are zero.
 *   SX      scale words as in mmac_gemm_dense_mx: ceil(K/128) x lds 32-bit
 *           words, byte q of SX[t*lds + i] is the exponent e (value 2^(e-127))
 *           of block 4t+q of row i.  lds >= M, 4-byte aligned (mmac_gemm_dense_mx
 *           itself asks for lds % 4 == 0 and 16 bytes), and the words span less
 *           than 2^31 bytes.  e = 255 stands for NaN: every
 *           element of that block is NaN to the calls below.
 */
#ifndef MMAC_LOWBIT_H
#define MMAC_LOWBIT_H

#include "mmac.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MMAC_U4 ((mmac_dtype_t)9)   /* unsigned 4-bit integer, two per byte */
#define MMAC_F32 ((mmac_dtype_t)10) /* IEEE binary32: inputs of the two quantizers, output of the dequantizer */

/* A w4 matrix (see above); host structure, read during the call only. */
typedef struct mmac_w4 {
    int32_t q_type;        /* MMAC_U4 or MMAC_FP4_E2M1 */
    int32_t group;         /* 32, 64, 128, or 0 for whole rows */
    void *codes;           /* N rows of 16*ceil(K/32) bytes */
    int64_t pitch;         /* bytes from one row of codes to the next */
    uint32_t *words;       /* scale words */
    int64_t ldw;           /* words from one group to the next */
} mmac_w4_t;

/*
 * Weights to 4 bits, round to nearest: W (w_type F16, BF16 or F32, row-major
 * N x K, ldw_in elements per row, 16-byte alignment and pitch) -> q.
 * Per group, with lo = min(0, w...) and hi = max(0, w...):
 *   U4, symmetric      r = max|w|,  s = r / 7,   z = 8
 *   U4, not symmetric  r = hi - lo, s = r / 15,  z = the integer nearest to -lo / s
 *   FP4 (symmetric must be 1)  r = max|w|, s = r / 6, z = 0
 * r and s are rounded to fp32 and s then to 16 significant bits; an s below
 * 2^-126 becomes 0 (then z is 8, 0 and 0, and every code is z).  The codes are
 * those nearest to w / s (+ z, then clamped to 0 .. 15), exact quotient, ties to
 * even.  A group that holds a NaN or an infinity, or whose r passes fp32, gets
 * the scale NaN and codes z (z = 8, 0, 0), so every product with it is NaN.
 * Code 0 fills the units past K.  N == 0 or K == 0: nothing is done.
 */
mmac_status_t mmac_w4_quantize(mmac_dtype_t w_type, int symmetric, int64_t N, int64_t K, const void *W,
                               int64_t ldw_in, const mmac_w4_t *q, void *stream);

/*
 * D = round(act(alpha * A*W + beta * C + bias)), W given as a w4 matrix (rows j =
 * columns of D): everything else as in mmac_gemm_dense_ep / _ws, with a_type F16
 * or BF16.  Sums and the scales are fp32: codes are exact in A's type, each
 * group's sum of a * (n - z) is scaled as a whole and added up in fp32, so the
 * weight itself is never rounded.  U4: that sum is formed as sum a*n - z * sum a
 * (an infinity in A can give NaN where (n - z) * a alone would be infinite).
 *   workspace  as in mmac_gemm_dense_ws (zeroed once, 16-byte aligned, shared by
 *              calls of any size and kind, but not by calls that may run at the
 *              same time); NULL, or smaller than
 *              mmac_gemm_w4_workspace_bytes says: the call runs unsplit.
 */
mmac_status_t mmac_gemm_w4(mmac_dtype_t a_type, int64_t M, int64_t N, int64_t K, double alpha, const void *A,
                           int64_t lda, const mmac_w4_t *W, double beta, const void *C, int64_t ldc, void *D,
                           int64_t ldd, const mmac_epilogue_t *ep, void *workspace, int64_t workspace_bytes,
                           void *stream);

/* Workspace bytes of mmac_gemm_w4 for this product (0: it would not split).  Host-only. */
int64_t mmac_gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Activations to an mx8 matrix: X (x_type F16, BF16 or F32, row-major M x K,
 * 16-byte alignment and pitch) -> Xq (q_type FP8_E4M3, BF8_E5M2 or I8) and SX.
 * Per block of 32 along K: e is the smallest exponent in 1 .. 254 (2^-126 and
 * up) for which max|x| <= T * 2^(e-127), T the type's largest value (448, 57344,
 * 127), and 127 for a block of zeros; each element is x * 2^(127-e) rounded to
 * nearest, ties to even.  Nothing saturates.  Non-finite elements: E4M3 stores
 * NaN for NaN and infinities, E5M2 keeps both, and neither counts towards the
 * block's maximum; an I8 block that holds one gets e = 255 and zero elements.
 * Exponents of blocks past K within the last word are 127.
 */
mmac_status_t mmac_mx8_quantize(mmac_dtype_t x_type, mmac_dtype_t q_type, int64_t M, int64_t K, const void *X,
                                int64_t ldx, void *Xq, int64_t ldq, uint32_t *SX, int64_t lds, void *stream);

/*
 * The reverse: X = Xq * 2^(e-127), rounded to x_type as the epilogues of mmac.h
 * round (to nearest, finite values saturate, F32 too: an element next to the largest
 * fp32 may have been rounded up past it).
 */
mmac_status_t mmac_mx8_dequantize(mmac_dtype_t q_type, mmac_dtype_t x_type, int64_t M, int64_t K, const void *Xq,
                                  int64_t ldq, const uint32_t *SX, int64_t lds, void *X, int64_t ldx, void *stream);

/*
 * Weight gradient of a linear layer from the saved 8-bit input: with dY the
 * M x N gradient of its output (y_type F16 or BF16, row-major) and the mx8 M x K
 * input (Xq, SX),
 *   D = alpha * dY^T * X + beta * C,   D and C row-major N x K.
 * The sum over the M rows is fp32.  X enters the products in dY's type: exact
 * for BF16 (every element times a power of two has at most 8 significant bits;
 * magnitudes below bf16's smallest subnormal round), rounded to binary16 for
 * F16 (exact in 2^-14 .. 65504).  Finite elements beyond the type's range
 * saturate, as in mmac_mx8_dequantize.
 *   ep         NULL, or d_type with act NONE and bias NULL
 *              (MMAC_ERR_UNSUPPORTED otherwise).
 *   workspace  as in mmac_gemm_dense_ws: M may be cut into ranges whose partial
 *              sums are added in range order (deterministic).
 * M == 0: D = beta * C.
 */
mmac_status_t mmac_gemm_mx8_wgrad(mmac_dtype_t y_type, mmac_dtype_t q_type, int64_t M, int64_t N, int64_t K,
                                  double alpha, const void *dY, int64_t ldy, const void *Xq, int64_t ldq,
                                  const uint32_t *SX, int64_t lds, double beta, const void *C, int64_t ldc, void *D,
                                  int64_t ldd, const mmac_epilogue_t *ep, void *workspace, int64_t workspace_bytes,
                                  void *stream);

/* Workspace bytes of mmac_gemm_mx8_wgrad for this product (0: it would not split).  Host-only. */
int64_t mmac_gemm_mx8_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* MMAC_LOWBIT_H */
