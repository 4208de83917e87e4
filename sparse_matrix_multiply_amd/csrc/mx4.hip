// Rows to 4-bit block-scaled elements (E2M1).
//
// A lane holds eight elements of a row and writes their eight codes, one word; an instruction of a wave covers 512
// columns of one row, a wave 8 rows, all loads in flight.  The scale words are column-major, so the workgroup's
// 32 words of one strip of 128 columns are one line: they are gathered in LDS.
//
// HBM bounds it: 16384 x 8192 bf16, 340 MB, in 56 us (6 TB/s, part of it from the last-level cache).  With all 8 rows' loads issued before the
// first is converted; the rows' ends cost no branch.
#include <algorithm>

#include "mx_block.h"
#include "rows.h"

namespace mmac {

// A workgroup's unit: 512 columns of 32 rows, 8 rows a wave.
constexpr int kRows = 32, kSteps = kRows / 4, kCols = 512;

template <int XT>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx8Params p, int64_t units, int blocks) {
    __shared__ uint32_t words[kCols / 128][kRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15;
    const int kp = (p.K + 31) / 32 * 32, strips = (p.K + 127) / 128;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int block = (int)(unit % blocks);
        const int64_t row0 = unit / blocks * kRows;
        const int e0 = block * kCols + lane * 8;
        Raw8<XT> x[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            x[s] = load_raw8<XT, kNonTemporal>(RowOf<XT>(p.X, row, p.x_pitch, row < p.M ? p.K : 0).whole, e0);
        }
        if ((p.K & 7) && block == blocks - 1) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int64_t row = row0 + wave * kSteps + s;
                if (e0 == (p.K & ~7) && row < p.M) RowOf<XT>(p.X, row, p.x_pitch, p.K).load_short(x[s], e0, p.K & 7);
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = row0 + wave * kSteps + s;
            float f[8], y[8];
            elements<XT>(x[s], f);
            bool odd;
            const int e = scale_block<DT_FP4>(f, y, odd);
            // the conversion rounds to nearest even and keeps zeros' signs; every |y| is at most 6
            uint32_t c = 0;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
            if (row < p.M && e0 < kp)
                *reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(p.Xq) + row * p.q_pitch + e0 / 2) = c;
            const uint32_t w = scale_word_of(e, l16);
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

template <int XT>
static hipError_t launch_as(const Mx8Params &p, hipStream_t s) {
    const int blocks = (p.K + kCols - 1) / kCols;
    const int64_t units = blocks * (((int64_t)p.M + kRows - 1) / kRows);
    hipLaunchKernelGGL(mx4_quantize_kernel<XT>, dim3((unsigned)std::min<int64_t>(units, 1 << 20)), dim3(256), 0, s, p, units,
                       blocks);
    return hipGetLastError();
}

hipError_t launch_mx4_quantize(int x, const Mx8Params &p, hipStream_t s) {
    switch (x) {
    case DT_F16: return launch_as<DT_F16>(p, s);
    case DT_BF16: return launch_as<DT_BF16>(p, s);
    case DT_F32: return launch_as<DT_F32>(p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mmac
