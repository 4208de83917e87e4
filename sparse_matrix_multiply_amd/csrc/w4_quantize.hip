// Weights to 4 bits with a scale word per group of a row.
//
// Per group: the range r of its values, the scale s = r / steps (fp32, then 16
// significant bits), the zero point z, and for each value the integer nearest to
// w / s, ties to even, of the exact quotient.  An fp32 quotient is rounded, so a
// value just off the middle between two integers could land on it: only there the
// sign of the exact remainder w - q * s (one fused multiply-add rounds once and
// keeps the sign) decides.
//
// The work is a streaming pass.  Groups of 32 to 128: a lane holds eight
// elements, 4 to 16 lanes a group, a wave 512 columns of 8 rows; the
// scale words (group-major) are gathered in LDS so that 32 consecutive ones are
// written at a time.  Whole rows: one workgroup per row reads the row twice, the
// second time from the caches.  A division per element would take longer than the
// memory does; the product with 1 / s (off by less than 4e-6 for quotients up
// to 15) decides everywhere but within 1e-5 of a middle.
//
// 8192^2 bf16 in groups of 128, not symmetric: 56 us (3.0 TB/s; 75 us with the
// division); whole rows 46 us.  A row's load branches on the row's end and is converted
// in the branch, so it is waited for before the next one is issued: what bounds
// the time is one load in flight per wave and, behind the loads, the vector
// instructions (about 13 per element, 22 us of issue), which overlap only with
// other waves' loads.  The E2M1 forms in groups of 64 and 128 keep one value in scratch.
#include <algorithm>

#include "lowbit.h"

namespace mmac {

// r / N correctly rounded: the product with the rounded reciprocal, corrected once by the remainder (checked
// for every significand with N = 6, 7 and 15).
template <int N>
__device__ __forceinline__ float divide_by(float r) {
    constexpr float inv = 1.0f / N;
    const float q = r * inv;
    return fmaf(fmaf(-(float)N, q, r), inv, q);
}

// The integer nearest to a / s (s > 0), ties to even, exact quotient.
__device__ __forceinline__ float nearest_quotient(float a, float s) {
    const float q = a / s, n = __builtin_rintf(q);
    if (__builtin_fabsf(q - n) == 0.5f) {
        const float rest = fmaf(-q, s, a);
        if (rest > 0.0f) return __builtin_ceilf(q);
        if (rest < 0.0f) return __builtin_floorf(q);
    }
    return n;
}

// Code of the E2M1 value nearest to a / s (a >= 0, s > 0), ties to the even code.
__device__ __forceinline__ uint32_t nearest_e2m1(float a, float s) {
    const float q = a / s;
    constexpr float middle[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        bool up = q > middle[i];
        if (q == middle[i]) {
            const float rest = fmaf(-q, s, a);
            up = rest > 0.0f || (rest == 0.0f && (i & 1));
        }
        code += up;
    }
    return code;
}

// Range of a group's values as fp32 bits, which order non-negative values as integers do.  Not symmetric: the
// largest value and the largest of the negated ones, both at least 0; else the largest magnitude.  A value that is
// not finite makes the largest one NaN or infinite.
template <bool SYM>
struct Range {
    uint32_t hi = 0, neg = 0;
    __device__ __forceinline__ void add(const float (&x)[8]) {
        if constexpr (SYM) {
#pragma unroll
            for (int i = 0; i < 8; ++i) hi = max(hi, __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu);
        } else {
            float h = __builtin_bit_cast(float, hi), l = -__builtin_bit_cast(float, neg), finite = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h = fmaxf(h, x[i]);
                l = fminf(l, x[i]);
                finite = fmaf(x[i], 0.0f, finite);   // NaN from a NaN or an infinity
            }
            hi = finite == 0.0f ? __builtin_bit_cast(uint32_t, h) : 0x7fc00000u;
            neg = __builtin_bit_cast(uint32_t, -l) & 0x7fffffffu;
        }
    }
    // over groups of LANES consecutive lanes, in every lane
    template <int LANES>
    __device__ __forceinline__ void gather() {
        const auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
        hi = reduce_lanes<LANES>(hi, larger);
        if constexpr (!SYM) neg = reduce_lanes<LANES>(neg, larger);
    }
    __device__ __forceinline__ float width() const {
        const float h = __builtin_bit_cast(float, hi);
        return SYM ? h : h + __builtin_bit_cast(float, neg);
    }
};

// How near to a middle between two codes a quotient formed with 1 / s may be believed.
constexpr float kNear = 1e-5f;

// The scale word, its scale and zero point, and about 1 / s.
template <int QT, bool SYM>
__device__ __forceinline__ uint32_t scale_word(const Range<SYM> &r, float &s, float &inv, float &z) {
    static_assert(SYM || QT != DT_FP4, "E2M1 codes have no zero point");
    s = divide_by<QT == DT_FP4 ? 6 : SYM ? 7 : 15>(r.width());
    inv = 0.0f;
    z = QT == DT_FP4 ? 0.0f : SYM ? 8.0f : 0.0f;
    uint32_t u = __builtin_bit_cast(uint32_t, s);
    if (u >= 0x7f800000u) {      // a NaN, an infinity, or a range past fp32
        s = 0.0f;
        return 0x7fc00000u | (uint32_t)z;
    }
    if (u < 0x00800000u) {
        s = 0.0f;
        return (uint32_t)z;
    }
    u = (u + 0x7fu + ((u >> 8) & 1u)) & ~0xffu;
    s = __builtin_bit_cast(float, u);
    inv = __builtin_amdgcn_rcpf(s);   // off by at most one unit of its last place
    if (QT != DT_FP4 && !SYM) {
        const float neg = __builtin_bit_cast(float, r.neg), q = neg * inv;
        float n = __builtin_rintf(q);
        if (__builtin_fabsf(q - n) > 0.5f - kNear) n = nearest_quotient(neg, s);
        z = fminf(fmaxf(n, 0.0f), 15.0f);
    }
    return u | (uint32_t)z;
}

// Code of x for scale s > 0, inv about 1 / s, before its sign, as a float; `off`: largest distance from a code.
template <int QT>
__device__ __forceinline__ float code_of(float x, float inv, float z, float &off) {
    if constexpr (QT == DT_FP4) {
        // steps of 1/2 below 2, of 1 below 4, of 2 above: in units of the step the code is the nearest integer plus 0, 2, 4
        const float a = __builtin_fabsf(x * inv);
        const float per = a < 2.0f ? 2.0f : a < 4.0f ? 1.0f : 0.5f, base = a < 2.0f ? 0.0f : a < 4.0f ? 2.0f : 4.0f;
        const float y = a * per, n = __builtin_rintf(y);
        off = fmaxf(off, __builtin_fabsf(y - n));
        return fminf(n + base, 7.0f);
    } else {
        // the integer nearest to x / s + z; z is whole, and ties are left to the exact code
        const float y = fmaf(x, inv, z), n = __builtin_rintf(y);
        off = fmaxf(off, __builtin_fabsf(y - n));
        return fminf(n, 15.0f);
    }
}
template <int QT>
__device__ __forceinline__ uint32_t exact_code(float x, float s, float z) {
    if constexpr (QT == DT_FP4) return nearest_e2m1(__builtin_fabsf(x), s) | (x < 0.0f ? 8u : 0u);
    else return (uint32_t)fminf(fmaxf(nearest_quotient(x, s) + z, 0.0f), 15.0f);
}

// Eight codes of a lane's elements e0 .. e0 + 7, those at and past K zero.
template <int QT>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float s, float inv, float z, int e0, int K) {
    uint32_t w = (uint32_t)z * 0x11111111u;   // s == 0: every code is z
    if (s != 0.0f) {
        float off = 0.0f;
        uint32_t even = 0, odd = 0;   // four codes each, a byte a code; the conversion stops at 0
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            even = __builtin_amdgcn_cvt_pk_u8_f32(code_of<QT>(x[2 * i], inv, z, off), i, even);
            odd = __builtin_amdgcn_cvt_pk_u8_f32(code_of<QT>(x[2 * i + 1], inv, z, off), i, odd);
        }
        w = even | (odd << 4);
        if constexpr (QT == DT_FP4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= x[i] < 0.0f ? 8u << (4 * i) : 0u;
        }
        if (!(off <= 0.5f - kNear)) {   // some quotient is too near a middle to tell
            w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= exact_code<QT>(x[i], s, z) << (4 * i);
        }
    }
    if (e0 + 8 > K) w = e0 >= K ? 0u : w & ((1u << (4 * (K - e0))) - 1u);
    return w;
}

// A workgroup's unit: 512 columns of 32 rows, 8 rows a wave; an instruction of a wave covers 512 columns of one row.
constexpr int kRows = 32, kSteps = kRows / 4, kCols = 512;

template <int WT, int QT, bool SYM, int GROUP>
__global__ __launch_bounds__(256, 4) void w4_quantize_kernel(W4QuantParams p, int64_t units, int blocks) {
    constexpr int LANES = GROUP / 8, PER = kCols / GROUP;   // lanes of a group, groups of a unit's row
    __shared__ uint32_t words[PER][kRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kp = (p.K + 31) / 32 * 32;
    const int groups = (p.K + GROUP - 1) / GROUP;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int block = (int)(unit % blocks);
        const int64_t row0 = unit / blocks * kRows;
        const int e0 = block * kCols + lane * 8;
        float x[kSteps][8];
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const int64_t row = row0 + wave * kSteps + st;
            load8<WT, true>(x[st], p.W + row * p.w_pitch, e0, row < p.N ? p.K : 0);
        }
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const int64_t row = row0 + wave * kSteps + st;
            Range<SYM> r;
            r.add(x[st]);
            r.template gather<LANES>();
            float s, inv, z;
            const uint32_t word = scale_word<QT, SYM>(r, s, inv, z);
            const uint32_t q = codes_of<QT>(x[st], s, inv, z, e0, p.K);
            if (row < p.N && e0 < kp) *reinterpret_cast<uint32_t *>(p.codes + row * p.pitch + e0 / 2) = q;
            if (lane % LANES == 0) words[lane / LANES][wave * kSteps + st] = word;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < PER * kRows; i += 256) {
            const int group = block * PER + i / kRows;
            const int64_t row = row0 + i % kRows;
            if (group < groups && row < p.N) p.words[group * p.ldw + row] = words[i / kRows][i % kRows];
        }
        __syncthreads();   // before the next unit's words
    }
}

template <int WT, int QT, bool SYM>
__global__ __launch_bounds__(256) void w4_quantize_rows_kernel(W4QuantParams p) {
    __shared__ uint32_t hi[4], neg[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kp = (p.K + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const uint8_t *src = p.W + row * p.w_pitch;
        Range<SYM> r;
        for (int64_t e0 = threadIdx.x * 8; e0 < p.K; e0 += 256 * 8) {
            float x[8];
            load8<WT>(x, src, e0, p.K);
            const uint32_t before = r.hi;
            r.add(x);
            r.hi = max(r.hi, before);   // a value that was not finite stays
        }
        for (int d = 1; d < 64; d *= 2) {
            r.hi = max(r.hi, (uint32_t)__shfl_xor((int)r.hi, d));
            r.neg = max(r.neg, (uint32_t)__shfl_xor((int)r.neg, d));
        }
        if (lane == 0) {
            hi[wave] = r.hi;
            neg[wave] = r.neg;
        }
        __syncthreads();
        for (int w = 0; w < 4; ++w) {
            r.hi = max(r.hi, hi[w]);
            r.neg = max(r.neg, neg[w]);
        }
        __syncthreads();   // before the next row's values
        float s, inv, z;
        const uint32_t word = scale_word<QT, SYM>(r, s, inv, z);
        if (threadIdx.x == 0) p.words[row] = word;
        for (int64_t e0 = threadIdx.x * 8; e0 < kp; e0 += 256 * 8) {
            float x[8];
            load8<WT>(x, src, e0, p.K);
            *reinterpret_cast<uint32_t *>(p.codes + row * p.pitch + e0 / 2) = codes_of<QT>(x, s, inv, z, (int)e0, p.K);
        }
    }
}

template <int WT, int QT, bool SYM>
static hipError_t launch_as(int group, const W4QuantParams &p, hipStream_t s) {
    if (group == 0) {
        hipLaunchKernelGGL((w4_quantize_rows_kernel<WT, QT, SYM>), dim3((unsigned)std::min(p.N, 1 << 20)), dim3(256), 0, s, p);
        return hipGetLastError();
    }
    const int blocks = (p.K + kCols - 1) / kCols;
    const int64_t units = blocks * (((int64_t)p.N + kRows - 1) / kRows);
    const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 20)), block(256);
    switch (group) {
    case 32: hipLaunchKernelGGL((w4_quantize_kernel<WT, QT, SYM, 32>), grid, block, 0, s, p, units, blocks); break;
    case 64: hipLaunchKernelGGL((w4_quantize_kernel<WT, QT, SYM, 64>), grid, block, 0, s, p, units, blocks); break;
    case 128: hipLaunchKernelGGL((w4_quantize_kernel<WT, QT, SYM, 128>), grid, block, 0, s, p, units, blocks); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}
template <int WT>
static hipError_t by_code(int q, bool sym, int group, const W4QuantParams &p, hipStream_t s) {
    if (q == DT_FP4) return launch_as<WT, DT_FP4, true>(group, p, s);
    return sym ? launch_as<WT, DT_U4, true>(group, p, s) : launch_as<WT, DT_U4, false>(group, p, s);
}

hipError_t launch_w4_quantize(int w, int q, bool sym, int group, const W4QuantParams &p, hipStream_t s) {
    switch (w) {
    case DT_F16: return by_code<DT_F16>(q, sym, group, p, s);
    case DT_BF16: return by_code<DT_BF16>(q, sym, group, p, s);
    case DT_F32: return by_code<DT_F32>(q, sym, group, p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mmac
