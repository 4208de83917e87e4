// Argument checks that the calls of mmac_lowbit.h, mmac_norm.h and mmac_grouped.h share.
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "launch.h"
#include "mmac_lowbit.h"

namespace mmac {

constexpr int64_t kMaxDim = 0x7fffffff;               // M, N, K below 2^31
constexpr int64_t kMaxPitchBytes = (int64_t)1 << 23;
constexpr int64_t kMaxWords = (((int64_t)1 << 31) - 1) / 4;   // words of a scale array

inline bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool bad_dim(int64_t n) { return n < 0 || n > kMaxDim; }
inline bool is_16bit(int t) { return t == MMAC_F16 || t == MMAC_BF16; }
inline bool is_mx8(int t) { return t == MMAC_I8 || t == MMAC_FP8_E4M3 || t == MMAC_BF8_E5M2; }
inline bool is_input(int t) { return is_16bit(t) || t == MMAC_F32; }
inline int elem_size(int t) { return t == MMAC_F32 ? 4 : is_16bit(t) ? 2 : 1; }
inline int out_size(int d_type) { return d_type == MMAC_OUT_ACC ? 4 : d_type <= MMAC_OUT_F16 ? 2 : 1; }

inline mmac_status_t launched(hipError_t e) { return e == hipSuccess ? MMAC_OK : MMAC_ERR_HIP; }

// A row-major operand of `cols` elements per row: leading dimension, pitch limit, alignment.
inline mmac_status_t check_rows(const void *p, int64_t ld, int64_t cols, int es) {
    if (ld < cols || ld < 1) return MMAC_ERR_INVALID_ARG;
    if (ld > kMaxPitchBytes / es) return MMAC_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || (ld * es) % 16) return MMAC_ERR_MISALIGNED;
    return MMAC_OK;
}

// The same of a matrix of `rows` rows: one without elements is not read, and its pitch says nothing.
inline mmac_status_t check_matrix(const void *p, int64_t ld, int64_t rows, int64_t cols, int es) {
    return rows == 0 || cols == 0 ? MMAC_OK : check_rows(p, ld, cols, es);
}

// A scale array of `rows` rows of ld words, `cols` of them used.
inline mmac_status_t check_words(const void *p, int64_t ld, int64_t rows, int64_t cols) {
    if (ld < cols || ld < 1) return MMAC_ERR_INVALID_ARG;
    if (rows > 0 && ld > kMaxWords / rows) return MMAC_ERR_UNSUPPORTED;
    if (!aligned(p, 4)) return MMAC_ERR_MISALIGNED;
    return MMAC_OK;
}

// alpha, beta, C, D and the epilogue of a floating product with an M x N output.
inline mmac_status_t check_out(int64_t M, int64_t N, double alpha, double beta, const void *C, int64_t ldc, const void *D,
                        int64_t ldd, const mmac_epilogue_t &ep) {
    if (ep.d_type < MMAC_OUT_ACC || ep.d_type > MMAC_OUT_BF8_E5M2 || ep.act < MMAC_ACT_NONE || ep.act > MMAC_ACT_RELU)
        return MMAC_ERR_INVALID_ARG;
    if ((M > 0 && N > 0 && (!D || (beta != 0.0 && !C))) || ldd < N || ldd < 1 || (beta != 0.0 && (ldc < N || ldc < 1))) return MMAC_ERR_INVALID_ARG;
    if (!std::isfinite(alpha) || !std::isfinite(beta) || std::fabs(alpha) > (double)FLT_MAX ||
        std::fabs(beta) > (double)FLT_MAX)
        return MMAC_ERR_INVALID_ARG;
    if (C == D && beta != 0.0 && ldc != ldd) return MMAC_ERR_INVALID_ARG;
    const int es = out_size(ep.d_type);
    if (ldd > kMaxPitchBytes / es || (beta != 0.0 && ldc > kMaxPitchBytes / es)) return MMAC_ERR_UNSUPPORTED;
    if (!aligned(D, es) || (beta != 0.0 && !aligned(C, es)) || (ep.bias && !aligned(ep.bias, 4))) return MMAC_ERR_MISALIGNED;
    return MMAC_OK;
}

inline mmac_epilogue_t epilogue_of(const mmac_epilogue_t *ep) {
    return ep ? *ep : mmac_epilogue_t{MMAC_OUT_ACC, MMAC_ACT_NONE, nullptr};
}

}  // namespace mmac
