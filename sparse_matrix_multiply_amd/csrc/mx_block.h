// Blocks of 32 consecutive elements of a row with one power-of-two scale 2^(e-127), as the kernels that write
// them form them: a lane holds eight elements, four lanes a block, sixteen lanes the 128 columns of a scale word.
//
// With T = c * 2^p (1 <= c < 2) the element type's largest value and m = max|x| = f * 2^r, the smallest exponent
// with m <= T * 2^(e-127) is r - p when f <= c and r - p + 1 otherwise; on m's fp32 bits both are one addition whose
// carry into the exponent field is exactly "f > c".  Scaling by a power of two is exact, so the only rounding
// is the one to the element type.
#pragma once

#include "lowbit.h"

namespace mmac {

template <int QT> struct MxType;
template <> struct MxType<DT_E4M3> { static constexpr int top = 8; static constexpr uint32_t frac = 0x600000; };
template <> struct MxType<DT_E5M2> { static constexpr int top = 15; static constexpr uint32_t frac = 0x600000; };
template <> struct MxType<DT_FP4> { static constexpr int top = 2; static constexpr uint32_t frac = 0x400000; };
template <> struct MxType<DT_I8> { static constexpr int top = 6; static constexpr uint32_t frac = 0x7e0000; };

// Eight scaled values -> eight element bytes.  The conversion instructions round to nearest even and are exact
// for the values met here (finite, at most the type's largest); a wave that holds a non-finite value takes the
// bit-level conversions.
template <int QT>
__device__ __forceinline__ u32x2 to_elements(const float (&y)[8], bool odd) {
    uint32_t w[2] = {0, 0};
    if constexpr (QT == DT_I8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)__builtin_rintf(y[i]) & 0xffu) << (8 * (i & 3));
    } else if (__any(odd)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t b;
            if constexpr (QT == DT_E4M3) {
                const uint32_t u = __builtin_bit_cast(uint32_t, y[i]);
                b = (u & 0x7fffffffu) >= 0x7f800000u ? ((u >> 24) & 0x80u) | 0x7fu : to_e4m3_sat(y[i]);
            } else {
                b = to_e5m2_sat(y[i]);
            }
            w[i / 4] |= b << (8 * (i & 3));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int v = 0;
            if constexpr (QT == DT_E4M3) {
                v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], v, false);
                v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], v, true);
            } else {
                v = __builtin_amdgcn_cvt_pk_bf8_f32(y[4 * h], y[4 * h + 1], v, false);
                v = __builtin_amdgcn_cvt_pk_bf8_f32(y[4 * h + 2], y[4 * h + 3], v, true);
            }
            w[h] = (uint32_t)v;
        }
    }
    return u32x2{w[0], w[1]};
}

// The exponent of this lane's block from its eight values x, and the scaled values y.  The largest magnitude is
// that of the finite elements (fp32 bits order like magnitudes); odd: this lane holds one that is not finite.
// Types without NaN (I8, FP4): a block that holds such an element gets e = 255 and zeros.
template <int QT>
__device__ __forceinline__ int scale_block(const float (&x)[8], float (&y)[8], bool &odd) {
    uint32_t m = 0, worst = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
        worst = max(worst, a);
        m = max(m, a >= 0x7f800000u ? 0u : a);
    }
    const auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
    m = reduce_lanes<4>(m, umax);
    odd = worst >= 0x7f800000u;
    int e = (int)((m + (0x7fffffu - MxType<QT>::frac)) >> 23) - MxType<QT>::top;
    e = m == 0 ? 127 : max(e, 1);   // at most 127 + 127 - 2 + 1
    const float scale = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * scale;
    if constexpr (QT == DT_I8 || QT == DT_FP4) {
        if (reduce_lanes<4>(worst, umax) >= 0x7f800000u) {
            e = 255;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        }
    }
    return e;
}

// The scale word of the sixteen lanes' row, in each of them: byte l16 / 4 from each group of four.
__device__ __forceinline__ uint32_t scale_word_of(int e, int l16) {
    uint32_t w = (uint32_t)e << (8 * (l16 >> 2));
    w |= dpp<kDppRor4>(w);
    w |= dpp<kDppRor8>(w);
    return w;
}

}  // namespace mmac
