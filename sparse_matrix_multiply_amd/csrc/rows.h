// Rows read and written eight elements per lane, without branches: whole groups of eight through a buffer
// descriptor that ends where they do (loads past it give zero, stores are dropped), so that all loads of a row can be in flight
// together; a row whose length is no multiple of eight has one more group, which its lane handles element by element.
#pragma once

#include "lowbit.h"

namespace mmac {

// Eight elements of type DT as they lie in memory.
template <int DT> struct Raw8 { i32x4 d[dt_size<DT>() / 2]; };

template <int DT, int POLICY>
__device__ __forceinline__ Raw8<DT> load_raw8(rsrc_t r, int e0) {
    Raw8<DT> x;
#pragma unroll
    for (int v = 0; v < dt_size<DT>() / 2; ++v)
        x.d[v] = __builtin_amdgcn_raw_buffer_load_b128(r, (uint32_t)e0 * dt_size<DT>() + 16 * v, 0, POLICY);
    return x;
}

// Element i of x, exact in fp32.
template <int DT>
__device__ __forceinline__ float element(const Raw8<DT> &x, int i) {
    if constexpr (DT == DT_F32) {
        const int w = x.d[i / 4][i % 4];
        return __builtin_bit_cast(float, w);
    } else {
        const uint32_t w = (uint32_t)x.d[0][i / 2];
        return from_out_bits<DT == DT_BF16 ? OUT_BF16 : OUT_F16>(i % 2 ? w >> 16 : w & 0xffffu);
    }
}
template <int DT>
__device__ __forceinline__ void elements(const Raw8<DT> &x, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = element<DT>(x, i);
}

// One element's bits, rounded to DT as the epilogues round (fp32: as it is).
template <int DT>
__device__ __forceinline__ uint32_t rounded(float f) {
    if constexpr (DT == DT_F32) return __builtin_bit_cast(uint32_t, f);
    else return DT == DT_BF16 ? to_bf16_sat(f) : to_f16_sat(f);
}
template <int DT>
__device__ __forceinline__ float from_bits(uint32_t b) {
    if constexpr (DT == DT_F32) return __builtin_bit_cast(float, b);
    else return from_out_bits<DT == DT_BF16 ? OUT_BF16 : OUT_F16>(b);
}
template <int DT>
__device__ __forceinline__ Raw8<DT> pack8(const float (&f)[8]) {
    Raw8<DT> x;
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.d[i / 4][i % 4] = (int)rounded<DT>(f[i]);
    } else {
        uint32_t o[4];
        pack16_sat<DT == DT_BF16 ? OUT_BF16 : OUT_F16>(f, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.d[0][i] = (int)o[i];
    }
    return x;
}

// A row of N elements of type DT.
template <int DT>
struct RowOf {
    uint8_t *at;
    rsrc_t whole;   // its whole groups of eight
    __device__ __forceinline__ RowOf(const void *base, int64_t row, int64_t pitch, int N)
        : at(const_cast<uint8_t *>(static_cast<const uint8_t *>(base)) + row * pitch),
          whole(make_rsrc(at, (uint32_t)(N & ~7) * dt_size<DT>())) {}
    // after load_raw8: the last, short group of a row (n = N mod 8 elements at e0), zeros behind it
    __device__ __forceinline__ void load_short(Raw8<DT> &x, int e0, int n) const {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = 0.0f;
            if (i < n) {
                if constexpr (DT == DT_F32) f[i] = reinterpret_cast<const float *>(at)[e0 + i];
                else f[i] = from_bits<DT>(reinterpret_cast<const uint16_t *>(at)[e0 + i]);
            }
        }
        // exact values: rounding keeps them; NaN becomes the quiet NaN
        x = pack8<DT>(f);
    }
    template <int POLICY>
    __device__ __forceinline__ void store(const Raw8<DT> &x, int e0) const {
#pragma unroll
        for (int v = 0; v < dt_size<DT>() / 2; ++v)
            __builtin_amdgcn_raw_buffer_store_b128(x.d[v], whole, (uint32_t)e0 * dt_size<DT>() + 16 * v, 0, POLICY);
    }
    __device__ __forceinline__ void store_short(const Raw8<DT> &x, int e0, int n) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) {
                if constexpr (DT == DT_F32) reinterpret_cast<uint32_t *>(at)[e0 + i] = (uint32_t)x.d[i / 4][i % 4];
                else reinterpret_cast<uint16_t *>(at)[e0 + i] = (uint16_t)((uint32_t)x.d[0][i / 2] >> (16 * (i % 2)));
            }
        }
    }
};

// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    const auto add = [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    };
    v = __builtin_bit_cast(float, reduce_lanes<16>(__builtin_bit_cast(uint32_t, v), add));
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}
// Sum over T threads (T / 64 consecutive waves of the workgroup; T = 64: no barrier).  `red` holds T / 64 words that
// no thread still reads.
template <int T>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += red[w];
    }
    return v;
}

// Rows (or units of rows) of one XCD: workgroups are dealt to the 8 XCDs round-robin, so XCD x takes the x-th
// contiguous part, and what neighbouring rows share (lines of the scale words) meets in one L2.  The grid is a multiple of 8.
struct XcdPart {
    int64_t first, count;
    __device__ __forceinline__ XcdPart(int64_t units) {
        const int x = blockIdx.x & 7;
        const int64_t q = units >> 3, r = units & 7;
        first = x * q + (x < r ? x : r);
        count = q + (x < r ? 1 : 0);
    }
};

}  // namespace mmac
