// Low-bit operands (include/mmac_lowbit.h): parameters of the kernels, their
// launchers, and the device primitives they share.
#pragma once

#include <type_traits>

#include "device.h"

namespace mmac {

// Type codes of mmac_lowbit.h beyond device.h's.
enum : int { DT_U4 = 9, DT_F32 = 10 };

// D = round(act(alpha * acc + beta * C + bias)) as the GEMMs of mmac.h have it.
struct OutParams {
    const void *C;
    int64_t ldc;
    void *D;
    int64_t ldd;
    float alpha, beta;
    int use_c;
    int d_type;          // OUT_*
    int act;
    const float *bias;   // NULL, or one per column of D
};

// Split sums: `splits` ranges of the summed axis, `per_split` chunks each; one
// counter per output tile (zero before and after every call), then the partial tiles.
struct SplitParams {
    int splits, per_split;
    uint32_t *counters;
    uint8_t *partials;
};

// Tiles of the 4-bit product for many rows, and elements of K per chunk.
enum W4Tile : int { W4_128x256, W4_128x128, W4_64x128 };
inline int w4_rows(W4Tile t) { return t == W4_64x128 ? 64 : 128; }
inline int w4_cols(W4Tile t) { return t == W4_128x256 ? 256 : 128; }
constexpr int kW4Chunk = 128;

struct W4Params {
    const uint8_t *A;
    int64_t a_pitch;     // bytes
    const uint8_t *codes;
    int64_t pitch;       // bytes
    const uint32_t *words;
    int64_t ldw;
    int groups;          // scale words of a row
    int group;           // 32, 64, 128 or 0 (whole rows)
    int M, N, K;
    W4Tile tile;            // tiled kernel
    int tiles_m, tiles_n;
    OutParams out;
    SplitParams split;
};

struct W4QuantParams {
    const uint8_t *W;
    int64_t w_pitch;     // bytes
    uint8_t *codes;
    int64_t pitch;
    uint32_t *words;
    int64_t ldw;
    int N, K;
};

struct Mx8Params {
    const uint8_t *X;    // the activations (written by the dequantizer)
    int64_t x_pitch;     // bytes
    const uint8_t *Xq;   // the elements (written by the quantizer)
    int64_t q_pitch;     // bytes
    const uint32_t *SX;
    int64_t lds;
    int M, K;
};

// Tiles of the weight gradient (rows: columns of dY; columns: of X) and rows of M per chunk.
enum WgradTile : int { WGRAD_32x128, WGRAD_64x128, WGRAD_128x128, WGRAD_256x256 };
inline int wgrad_rows(WgradTile t) {
    return t == WGRAD_32x128 ? 32 : t == WGRAD_64x128 ? 64 : t == WGRAD_128x128 ? 128 : 256;
}
inline int wgrad_cols(WgradTile t) { return t == WGRAD_256x256 ? 256 : 128; }
constexpr int kWgradChunk = 64;

struct WgradParams {
    const uint8_t *Y;
    int64_t y_pitch;     // bytes
    const uint8_t *Xq;
    int64_t q_pitch;     // bytes
    const uint32_t *SX;
    int64_t lds;
    int M, N, K;
    WgradTile tile;
    int tiles_n, tiles_k;
    OutParams out;
    SplitParams split;
};

hipError_t launch_w4_quantize(int w_type, int q_type, bool symmetric, int group, const W4QuantParams &p, hipStream_t s);
hipError_t launch_gemm_w4_rows(int a_type, int q_type, const W4Params &p, hipStream_t s);
hipError_t launch_gemm_w4_tiled(int a_type, int q_type, const W4Params &p, hipStream_t s);
hipError_t launch_mx8_quantize(int x_type, int q_type, const Mx8Params &p, hipStream_t s);
hipError_t launch_mx8_dequantize(int q_type, int x_type, const Mx8Params &p, hipStream_t s);
hipError_t launch_mx4_quantize(int x_type, const Mx8Params &p, hipStream_t s);   // Xq: packed codes
hipError_t launch_gemm_mx8_wgrad(int y_type, int q_type, const WgradParams &p, hipStream_t s);

#if defined(__HIPCC__)

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT> constexpr int dt_size() { return DT == DT_F32 ? 4 : DT == DT_F16 || DT == DT_BF16 ? 2 : 1; }

// Eight consecutive elements of a row of type DT, from element e0, as fp32; those at and past `limit` zero.
// STREAM: read past the caches' retention (data that no one reads again; 8192^2 bf16 quantized 5 % faster).
template <int DT, bool STREAM = false>
__device__ __forceinline__ void load8(float (&x)[8], const uint8_t *row, int64_t e0, int64_t limit) {
    constexpr int ES = dt_size<DT>();
    if (e0 + 8 <= limit) {
        uint32_t w[2 * ES];
#pragma unroll
        for (int v = 0; v < ES / 2; ++v) {
            const i32x4 *at = reinterpret_cast<const i32x4 *>(row + e0 * ES) + v;
            const i32x4 d = STREAM ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * v + i] = (uint32_t)d[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == DT_F32) x[i] = __builtin_bit_cast(float, w[i]);
            else x[i] = from_out_bits<DT == DT_BF16 ? OUT_BF16 : OUT_F16>((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = 0.0f;
            if (e0 + i < limit) {
                if constexpr (DT == DT_F32) x[i] = reinterpret_cast<const float *>(row)[e0 + i];
                else x[i] = from_out_bits<DT == DT_BF16 ? OUT_BF16 : OUT_F16>(reinterpret_cast<const uint16_t *>(row)[e0 + i]);
            }
        }
    }
}

// 32 x 32 tile, 16 elements of the summed axis.
template <int DT>
__device__ __forceinline__ f32x16 mma32(const i32x4 &a, const i32x4 &b, f32x16 c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Lane permutations within 16 lanes (data-parallel primitives, no LDS).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140, kDppRor4 = 0x124, kDppRor8 = 0x128;

// op over groups of LANES consecutive lanes (4, 8 or 16), the result in every lane.
template <int LANES, class F>
__device__ __forceinline__ uint32_t reduce_lanes(uint32_t v, F op) {
    v = op(v, dpp<kDppXor1>(v));
    v = op(v, dpp<kDppXor2>(v));
    if constexpr (LANES >= 8) v = op(v, dpp<kDppMirror8>(v));
    if constexpr (LANES >= 16) v = op(v, dpp<kDppMirror16>(v));
    return v;
}

// Every LDS access of this wave has completed; outstanding memory loads may remain.
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}

// One output element of a floating product: row i, column j, from its fp32 sum.
__device__ __forceinline__ void store_out(const OutParams &o, int64_t i, int64_t j, float acc) {
    float v = o.alpha * acc;
    const bool has_bias = o.bias != nullptr, relu = o.act != 0;
    const float bias = has_bias ? o.bias[j] : 0.0f;
    if (o.d_type == OUT_ACC) {
        if (o.use_c) v = fmaf(o.beta, static_cast<const float *>(o.C)[i * o.ldc + j], v);
        static_cast<uint32_t *>(o.D)[i * o.ldd + j] = finish<OUT_ACC>(v, bias, has_bias, relu);
    } else if (o.d_type <= OUT_F16) {
        const uint16_t *c = static_cast<const uint16_t *>(o.C) + (o.use_c ? i * o.ldc + j : 0);
        uint16_t *d = static_cast<uint16_t *>(o.D) + i * o.ldd + j;
        if (o.d_type == OUT_BF16) {
            if (o.use_c) v = fmaf(o.beta, from_out_bits<OUT_BF16>(*c), v);
            *d = (uint16_t)finish<OUT_BF16>(v, bias, has_bias, relu);
        } else {
            if (o.use_c) v = fmaf(o.beta, from_out_bits<OUT_F16>(*c), v);
            *d = (uint16_t)finish<OUT_F16>(v, bias, has_bias, relu);
        }
    } else {
        const uint8_t *c = static_cast<const uint8_t *>(o.C) + (o.use_c ? i * o.ldc + j : 0);
        uint8_t *d = static_cast<uint8_t *>(o.D) + i * o.ldd + j;
        if (o.d_type == OUT_E4M3) {
            if (o.use_c) v = fmaf(o.beta, from_out_bits<OUT_E4M3>(*c), v);
            *d = (uint8_t)finish<OUT_E4M3>(v, bias, has_bias, relu);
        } else {
            if (o.use_c) v = fmaf(o.beta, from_out_bits<OUT_E5M2>(*c), v);
            *d = (uint8_t)finish<OUT_E5M2>(v, bias, has_bias, relu);
        }
    }
}

// A 32 x 32 accumulator tile to rows row0 .. row0 + 31 and column j of D (lane L: column L mod 32, register e: row
// 8 (e / 4) + 4 (L / 32) + e mod 4); rows at and past `rows` and lanes with `in` false are left out.  All of C
// is read before D is written, so that its 16 reads are in flight together (C may be D).
template <int OT>
__device__ __forceinline__ void store_tile(const OutParams &o, int64_t row0, int rows, int64_t j, bool in, const f32x16 &acc) {
    typedef std::conditional_t<OT == OUT_ACC, uint32_t, std::conditional_t<OT <= OUT_F16, uint16_t, uint8_t>> T;
    const int first = (threadIdx.x & 32) / 8;
    const bool has_bias = o.bias != nullptr, relu = o.act != 0;
    if (!in) return;
    const float bias = has_bias ? o.bias[j] : 0.0f;
    T c[16] = {};
    if (o.use_c) {
        const T *C = static_cast<const T *>(o.C) + row0 * o.ldc + j;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int r = first + 8 * (e / 4) + e % 4;
            if (r < rows) c[e] = C[r * o.ldc];
        }
    }
    T *D = static_cast<T *>(o.D) + row0 * o.ldd + j;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int r = first + 8 * (e / 4) + e % 4;
        float v = o.alpha * acc[e];
        if (o.use_c) v = fmaf(o.beta, from_out_bits<OT>(c[e]), v);
        if (r < rows) D[r * o.ldd] = (T)finish<OT>(v, bias, has_bias, relu);
    }
}
// body(integral constant of D's type), so that the choice is made once for all of a wave's tiles.
template <class F>
__device__ __forceinline__ void by_out_type(int d_type, F body) {
    switch (d_type) {
    case OUT_ACC: return body(std::integral_constant<int, OUT_ACC>{});
    case OUT_BF16: return body(std::integral_constant<int, OUT_BF16>{});
    case OUT_F16: return body(std::integral_constant<int, OUT_F16>{});
    case OUT_E4M3: return body(std::integral_constant<int, OUT_E4M3>{});
    default: return body(std::integral_constant<int, OUT_E5M2>{});
    }
}

#endif  // __HIPCC__

}  // namespace mmac
