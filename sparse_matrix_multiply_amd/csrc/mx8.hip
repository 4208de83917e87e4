// 8-bit block-scaled activations: the quantizer and the dequantizer.
//
// A block is 32 consecutive elements of a row with one power-of-two scale,
// 2^(e-127).  With T = c * 2^p (1 <= c < 2) the element type's largest value and
// m = max|x| = f * 2^r, the smallest exponent with m <= T * 2^(e-127) is r - p
// when f <= c and r - p + 1 otherwise; on m's fp32 bits both are one addition
// whose carry into the exponent field is exactly "f > c".  Scaling by a power of
// two is exact, so the only rounding is the one to the element type.
//
// Both kernels stream, so HBM sets their time.  A lane holds eight elements of
// a row (16 bytes of a 16-bit type), four lanes a block, sixteen lanes the 128
// columns of one scale word; an instruction of a wave covers 512 columns of one
// row (1 KiB of a 16-bit type), a wave 8 rows: in the dequantizer with all their loads
// in flight, in the quantizer one after the other (each load branches on the row's end
// and is converted in the branch), so that many waves have to cover the latency.
// Scale words are stored column-major (one 128-column strip after the other), so
// the workgroup's 32 words of one strip are one 128-byte line: the quantizer
// gathers them in LDS and writes whole lines.  8192^2 bf16 and E4M3: quantized in 43 us
// (4.7 TB/s), restored in 43 us (4.8 TB/s), where a copy moves 4.9 to 5.5 TB/s; in strips of 128
// columns of 4 rows per instruction the quantizer took 50 us.
#include <algorithm>

#include "lowbit.h"

namespace mmac {

// A workgroup's unit: 512 columns of 32 rows, 8 rows a wave.
constexpr int kRows = 32, kSteps = kRows / 4, kCols = 512;

template <int QT> struct Mx8Type;
template <> struct Mx8Type<DT_E4M3> { static constexpr int top = 8; static constexpr uint32_t frac = 0x600000; };
template <> struct Mx8Type<DT_E5M2> { static constexpr int top = 15; static constexpr uint32_t frac = 0x600000; };
template <> struct Mx8Type<DT_I8> { static constexpr int top = 6; static constexpr uint32_t frac = 0x7e0000; };

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

template <int XT, int QT>
__global__ __launch_bounds__(256) void mx8_quantize_kernel(Mx8Params p, int64_t units, int blocks) {
    __shared__ uint32_t words[kCols / 128][kRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
    const int kp = (p.K + 31) / 32 * 32, strips = (p.K + 127) / 128;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int block = (int)(unit % blocks);
        const int64_t row0 = unit / blocks * kRows;
        const int e0 = block * kCols + lane * 8;
        float x[kSteps][8];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            load8<XT, true>(x[s], p.X + row * p.x_pitch, e0, row < p.M ? p.K : 0);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            // largest magnitude (fp32 bits order like magnitudes) over the finite elements, and whether all are
            uint32_t m = 0, worst = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t a = __builtin_bit_cast(uint32_t, x[s][i]) & 0x7fffffffu;
                worst = max(worst, a);
                m = max(m, a >= 0x7f800000u ? 0u : a);
            }
            const auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
            m = reduce_lanes<4>(m, umax);
            bool odd = worst >= 0x7f800000u;
            int e = (int)((m + (0x7fffffu - Mx8Type<QT>::frac)) >> 23) - Mx8Type<QT>::top;
            e = m == 0 ? 127 : max(e, 1);   // at most 127 + 127 - 6 + 1
            const float scale = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[s][i] * scale;
            if constexpr (QT == DT_I8) {
                if (reduce_lanes<4>(worst, umax) >= 0x7f800000u) {
                    e = 255;
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
                }
            }
            const u32x2 q = to_elements<QT>(y, odd);
            if (row < p.M && e0 < kp)
                *reinterpret_cast<u32x2 *>(const_cast<uint8_t *>(p.Xq) + row * p.q_pitch + e0) = q;
            // the word of this row: byte l16 / 4 from each group of four lanes
            uint32_t w = (uint32_t)e << (8 * (l16 >> 2));
            w |= dpp<kDppRor4>(w);
            w |= dpp<kDppRor8>(w);
            if (l16 == 0) words[lane >> 4][wave * kSteps + s] = w;
        }
        __syncthreads();
        if (threadIdx.x < kCols / 128 * kRows) {
            const int strip = block * (kCols / 128) + threadIdx.x / kRows;
            const int64_t row = row0 + threadIdx.x % kRows;
            if (strip < strips && row < p.M)
                const_cast<uint32_t *>(p.SX)[strip * p.lds + row] = words[threadIdx.x / kRows][threadIdx.x % kRows];
        }
        __syncthreads();   // before the next unit's words
    }
}

template <int QT, int XT>
__global__ __launch_bounds__(256) void mx8_dequantize_kernel(Mx8Params p, int64_t units, int blocks) {
    constexpr int ES = dt_size<XT>();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
    const int kp = (p.K + 31) / 32 * 32;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int block = (int)(unit % blocks), strip = block * (kCols / 128) + (lane >> 4);
        const int64_t row0 = unit / blocks * kRows;
        const int e0 = block * kCols + lane * 8;
        u32x2 q[kSteps];
        uint32_t w[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            const bool in = row < p.M && e0 < kp;
            // read past the caches' retention; the result is left in them for who asked for it
            q[s] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p.Xq + row * p.q_pitch + e0)) : u32x2{0, 0};
            w[s] = in ? p.SX[strip * p.lds + row] : 0;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            const uint32_t e = (w[s] >> (8 * (l16 >> 2))) & 255u;
            const float scale = __builtin_bit_cast(float, e == 255 ? 0x7fc00000u : e == 0 ? 0x00400000u : e << 23);
            float v[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int d = (int)q[s][h];
                if constexpr (QT == DT_I8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[4 * h + i] = (float)(int8_t)(d >> (8 * i));
                } else if constexpr (QT == DT_E4M3) {
                    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(d, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(d, true);
                    v[4 * h] = a[0]; v[4 * h + 1] = a[1]; v[4 * h + 2] = b[0]; v[4 * h + 3] = b[1];
                } else {
                    const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(d, false), b = __builtin_amdgcn_cvt_pk_f32_bf8(d, true);
                    v[4 * h] = a[0]; v[4 * h + 1] = a[1]; v[4 * h + 2] = b[0]; v[4 * h + 3] = b[1];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
            if (e >= 240 && e < 255) {   // products past fp32's range saturate; E5M2's own infinities stay
                constexpr float kMax = 3.40282347e38f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool inf_code = QT == DT_E5M2 && ((q[s][i / 4] >> (8 * (i & 3))) & 0x7fu) == 0x7cu;
                    if (__builtin_isinf(v[i]) && !inf_code) v[i] = __builtin_copysignf(kMax, v[i]);
                }
            }
            uint32_t o[2 * ES] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = v[i];
                if constexpr (XT == DT_F32) o[i] = __builtin_bit_cast(uint32_t, f);
                else o[i / 2] |= (XT == DT_BF16 ? to_bf16_sat(f) : to_f16_sat(f)) << (16 * (i & 1));
            }
            if (row >= p.M) continue;
            uint8_t *dst = const_cast<uint8_t *>(p.X) + row * p.x_pitch + (int64_t)e0 * ES;
            if (e0 + 8 <= p.K) {
#pragma unroll
                for (int u = 0; u < ES / 2; ++u)
                    reinterpret_cast<i32x4 *>(dst)[u] = i32x4{(int)o[4 * u], (int)o[4 * u + 1], (int)o[4 * u + 2], (int)o[4 * u + 3]};
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e0 + i < p.K) {
                        if constexpr (ES == 4) reinterpret_cast<uint32_t *>(dst)[i] = o[i];
                        else reinterpret_cast<uint16_t *>(dst)[i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
                    }
            }
        }
    }
}

// Workgroups over units; what the grid does not hold at once they walk over.
template <class K>
static hipError_t launch_units(K kernel, const Mx8Params &p, hipStream_t s) {
    const int blocks = (p.K + kCols - 1) / kCols;
    const int64_t units = blocks * (((int64_t)p.M + kRows - 1) / kRows);
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(units, 1 << 20)), dim3(256), 0, s, p, units, blocks);
    return hipGetLastError();
}
template <int XT, int QT>
static hipError_t quantize_as(const Mx8Params &p, hipStream_t s) {
    return launch_units(mx8_quantize_kernel<XT, QT>, p, s);
}
template <int XT, int QT>
static hipError_t dequantize_as(const Mx8Params &p, hipStream_t s) {
    return launch_units(mx8_dequantize_kernel<QT, XT>, p, s);
}

template <int XT>
static hipError_t by_element(int q, bool back, const Mx8Params &p, hipStream_t s) {
    switch (q) {
    case DT_E4M3: return back ? dequantize_as<XT, DT_E4M3>(p, s) : quantize_as<XT, DT_E4M3>(p, s);
    case DT_E5M2: return back ? dequantize_as<XT, DT_E5M2>(p, s) : quantize_as<XT, DT_E5M2>(p, s);
    case DT_I8: return back ? dequantize_as<XT, DT_I8>(p, s) : quantize_as<XT, DT_I8>(p, s);
    default: return hipErrorInvalidValue;
    }
}
static hipError_t by_type(int x, int q, bool back, const Mx8Params &p, hipStream_t s) {
    switch (x) {
    case DT_F16: return by_element<DT_F16>(q, back, p, s);
    case DT_BF16: return by_element<DT_BF16>(q, back, p, s);
    case DT_F32: return by_element<DT_F32>(q, back, p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mx8_quantize(int x, int q, const Mx8Params &p, hipStream_t s) { return by_type(x, q, false, p, s); }
hipError_t launch_mx8_dequantize(int q, int x, const Mx8Params &p, hipStream_t s) { return by_type(x, q, true, p, s); }

}  // namespace mmac
