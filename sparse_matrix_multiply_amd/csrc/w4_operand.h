// 4-bit codes to matrix-instruction operands.
//
// The byte 0x0n read as E4M3 is n * 2^-9 for every n from 0 to 15 (subnormals up
// to 7, then the first normal binade), so the instructions that convert pairs of
// fp8 values with a power-of-two scale give n exactly; E2M1 codes have a
// conversion of their own.
#pragma once

#include "lowbit.h"

namespace mmac {

// Eight codes of a word, ascending, as a 16-byte operand of DT values.
template <int DT, int QT>
__device__ __forceinline__ i32x4 operand_of(uint32_t w) {
    i32x4 f;
    if constexpr (QT == DT_FP4) {
        if constexpr (DT == DT_BF16) {
            f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
            f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
            f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
            f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
        } else {
            f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
            f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
            f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
            f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
        }
    } else {
        const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
        // bytes in ascending order: n0 n1 n2 n3 and n4 n5 n6 n7
        const uint32_t p0 = __builtin_amdgcn_perm(odd, even, 0x05010400u), p1 = __builtin_amdgcn_perm(odd, even, 0x07030602u);
        if constexpr (DT == DT_BF16) {
            f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, false));
            f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, true));
            f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, false));
            f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, true));
        } else {
            f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p0, 512.0f, false));
            f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p0, 512.0f, true));
            f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p1, 512.0f, false));
            f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p1, 512.0f, true));
        }
    }
    return f;
}

}  // namespace mmac
