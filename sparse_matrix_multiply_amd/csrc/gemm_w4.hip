// Products with 4-bit weights and group scales, few rows: D = A * W with W
// streamed once as codes.
//
// With codes n, zero point z and scale s per group g of a weight row j,
//   sum_k a_ik (n_jk - z_jg) s_jg = sum_g s_jg ( sum_{k in g} a_ik n_jk - z_jg sum_{k in g} a_ik ).
// Codes 0 .. 15 (and E2M1 values) are exact in bf16 and fp16, so the inner sums run on
// the 16 x 16 matrix instructions with no rounding of the weight: one
// accumulator starts at zero in every group, a second one sums A itself (an
// operand of ones), and at the group's end s * (t - z * u) joins the fp32 total.
//
// A workgroup owns 16 columns of D and all rows (up to 32); its WK waves split K
// into contiguous ranges of chunks of 256 elements: of a weight row one 128-byte
// line, of A 512 bytes.  Each wave copies a chunk straight into LDS, in whole
// lines, reads the fragments from there into registers and has the next chunk
// copied while it multiplies; no barrier until the partial tiles are added up in
// wave order.  The time is that of streaming the codes from HBM, and what covers
// the latency is many workgroups per compute unit rather than many chunks per
// wave: with one chunk per wave in LDS instead of two to four, 1 x 8192 x 8192 (U4,
// groups of 128) takes 8.8 us instead of 13.1 (4.0 TB/s), 16 rows 11.9 instead of
// 15.9, 4 x 32768 x 8192 (E2M1, groups of 32) 37.5 instead of 50 (4.5 TB/s).  From a few
// rows on A counts too: every workgroup of 16 columns reads all of it (16 bits an
// element, 13 x 10250 x 4100: 68 MB in all, from the caches, beside 21 MB of codes).
#include "gemm_tiled.h"
#include "w4_operand.h"

namespace mmac {

template <int DT>
__device__ __forceinline__ f32x4 mma16(const i32x4 &a, const i32x4 &b, f32x4 c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// MR rows of A are staged (2, 4, 8, 16 or 32, at least the rows there are); lanes of
// further rows read staged ones again, and their results are not stored.
// GROUP 128 also serves whole rows (every chunk then reads word 0).
template <int DT, int QT, int GROUP, int MR, int WK>
__global__ __launch_bounds__(WK * 64) void gemm_w4_rows_kernel(W4Params p) {
    constexpr int MB = MR > 16 ? 2 : 1;
    constexpr int GPC = 256 / GROUP;              // groups of a chunk
    constexpr int SPG = GROUP / 32;               // instruction steps of a group
    constexpr int SI = (GPC * 16 + 63) / 64;      // copy instructions for scale words
    constexpr int W_BYTES = 16 * 128, A_BYTES = MR * 512, SLOT = W_BYTES + A_BYTES + SI * 256;
    constexpr int OUTS = MB * 256;
    constexpr int RED = WK * OUTS * 4;
    constexpr int LDS_BYTES = WK * SLOT > RED ? WK * SLOT : RED;
    static_assert(LDS_BYTES <= 80 * 1024, "LDS: at least two workgroups per compute unit");
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
    const int col0 = blockIdx.x * 16, rows = p.M;
    const int cols = min(16, p.N - col0);
    const int row_bytes = (p.K + 31) / 32 * 16;
    const rsrc_t ra = make_rsrc(p.A, (uint32_t)(rows * p.a_pitch));
    const rsrc_t rw = make_rsrc(p.codes + (int64_t)col0 * p.pitch, (uint32_t)((cols - 1) * p.pitch + row_bytes));
    const rsrc_t rs = make_rsrc(p.words + col0, (uint32_t)(((p.groups - 1) * p.ldw + cols) * 4));

    f32x4 acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int nfull = p.K / 256, nall = (p.K + 255) / 256;
    const int per = (nall + WK - 1) / WK;
    const int c0 = min(wave * per, nall), c1 = min(c0 + per, nall), c1f = min(c1, nfull);
    uint8_t *slot = smem + wave * SLOT;

    const auto issue_w = [&](int c) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // 8 rows x one line; unit u of row r at u ^ ((r / 2) mod 8)
            const int r = 8 * j + (lane >> 3);
            const uint32_t unit = (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(slot + j * 1024), 16,
                                                     (uint32_t)r * (uint32_t)p.pitch + (uint32_t)c * 128u + unit * 16u, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < SI; ++j) {   // 4 groups x 16 columns of words
            const int d = j * 64 + lane, g = p.group == 0 ? 0 : c * GPC + (d >> 4);
            const uint32_t off = d < GPC * 16 && g < p.groups ? (uint32_t)((g * p.ldw + (d & 15)) * 4) : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(slot + W_BYTES + A_BYTES + j * 256), 4, off, 0, 0, 0);
        }
    };
    // unit u (8 elements) of row r of A sits at unit u ^ (r mod 16): 16 rows' reads of one unit meet 16 bank groups
    const auto issue_a = [&](int c) {
#pragma unroll
        for (int j = 0; j < MR / 2; ++j) {
            const int r = 2 * j + (lane >> 5);
            const uint32_t unit = (uint32_t)((lane & 31) ^ (r & 15));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(slot + W_BYTES + j * 1024), 16,
                                                     (uint32_t)r * (uint32_t)p.a_pitch + (uint32_t)c * 512u + unit * 16u, 0, 0, 0);
        }
    };
    constexpr int kOne = DT == DT_BF16 ? 0x3f803f80 : 0x3c003c00;
    const i32x4 ones = {kOne, kOne, kOne, kOne};

    uint32_t wd[8], sw[GPC];
    i32x4 a[8][MB];
    const auto load = [&]() {
#pragma unroll
        for (int v = 0; v < 8; ++v) {   // step v: elements 32 v + 8 q .. + 7 of the chunk
            wd[v] = *reinterpret_cast<const uint32_t *>(slot + r16 * 128 + ((v ^ ((r16 >> 1) & 7)) << 4) + q * 4);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int r = (m * 16 + r16) % MR;
                a[v][m] = *reinterpret_cast<const i32x4 *>(slot + W_BYTES + r * 512 + (((4 * v + q) ^ (r & 15)) << 4));
            }
        }
#pragma unroll
        for (int g = 0; g < GPC; ++g)
            sw[g] = *reinterpret_cast<const uint32_t *>(slot + W_BYTES + A_BYTES + (g * 16 + r16) * 4);
    };
    const auto compute = [&]() {
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < GPC; ++g) {
            f32x4 t[MB], u[MB];
#pragma unroll
            for (int v = g * SPG; v < (g + 1) * SPG; ++v) {
                const i32x4 b = operand_of<DT, QT>(wd[v]);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    t[m] = mma16<DT>(a[v][m], b, v == g * SPG ? zero : t[m]);
                    if constexpr (QT == DT_U4) u[m] = mma16<DT>(a[v][m], ones, v == g * SPG ? zero : u[m]);
                }
            }
            const float s = __builtin_bit_cast(float, sw[g] & ~0xffu), z = (float)(sw[g] & 0xffu);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = t[m][i];
                    if constexpr (QT == DT_U4) x = fmaf(-z, u[m][i], x);
                    acc[m][i] = fmaf(s, x, acc[m][i]);
                }
        }
    };

    if (c0 < c1f) {
        issue_w(c0);
        issue_a(c0);
    }
    for (int c = c0; c < c1f; ++c) {
        wait_vm_lgkm0<0>();   // chunk c has landed
        load();
        wait_lds();           // read before it is copied over
        if (c + 1 < c1f) {
            issue_w(c + 1);
            issue_a(c + 1);
        }
        compute();
    }
    if (c0 < c1 && c1 > nfull) {   // the chunk K ends inside: A through registers, zero past K (codes there are finite)
        issue_w(c1f);
        for (int j = 0; j < MR / 2; ++j) {
            const int r = 2 * j + (lane >> 5), unit = lane & 31, e0 = c1f * 256 + unit * 8;
            *reinterpret_cast<i32x4 *>(slot + W_BYTES + r * 512 + ((unit ^ (r & 15)) << 4)) =
                masked_unit<2>(ra, (uint32_t)r * (uint32_t)p.a_pitch + (uint32_t)e0 * 2u, e0, p.K);
        }
        wait_vm_lgkm0<0>();
        load();
        compute();
    }

    // add the partial tiles in wave order
    __syncthreads();
    float(*red)[MB][4][64] = reinterpret_cast<float(*)[MB][4][64]>(smem);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][m][i][lane] = acc[m][i];
    __syncthreads();
    for (int o = threadIdx.x; o < OUTS; o += WK * 64) {
        const int l = o & 63, i = (o >> 6) & 3, m = o >> 8;
        const int row = m * 16 + 4 * (l >> 4) + i, col = l & 15;
        float v = red[0][m][i][l];
        for (int w = 1; w < WK; ++w) v += red[w][m][i][l];
        if (row < rows && col < cols) store_out(p.out, row, col0 + col, v);
    }
}

template <int DT, int QT, int GROUP>
static hipError_t launch_rows(const W4Params &p, hipStream_t s) {
    const dim3 grid((p.N + 15) / 16);
    if (p.M <= 2) hipLaunchKernelGGL((gemm_w4_rows_kernel<DT, QT, GROUP, 2, 8>), grid, dim3(512), 0, s, p);
    else if (p.M <= 4) hipLaunchKernelGGL((gemm_w4_rows_kernel<DT, QT, GROUP, 4, 8>), grid, dim3(512), 0, s, p);
    else if (p.M <= 8) hipLaunchKernelGGL((gemm_w4_rows_kernel<DT, QT, GROUP, 8, 4>), grid, dim3(256), 0, s, p);
    else if (p.M <= 16) hipLaunchKernelGGL((gemm_w4_rows_kernel<DT, QT, GROUP, 16, 4>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gemm_w4_rows_kernel<DT, QT, GROUP, 32, 4>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}
template <int DT, int QT>
static hipError_t by_group(const W4Params &p, hipStream_t s) {
    switch (p.group) {
    case 32: return launch_rows<DT, QT, 32>(p, s);
    case 64: return launch_rows<DT, QT, 64>(p, s);
    case 0:
    case 128: return launch_rows<DT, QT, 128>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gemm_w4_rows(int a, int q, const W4Params &p, hipStream_t s) {
    if (a == DT_BF16) return q == DT_FP4 ? by_group<DT_BF16, DT_FP4>(p, s) : by_group<DT_BF16, DT_U4>(p, s);
    if (a == DT_F16) return q == DT_FP4 ? by_group<DT_F16, DT_FP4>(p, s) : by_group<DT_F16, DT_U4>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
