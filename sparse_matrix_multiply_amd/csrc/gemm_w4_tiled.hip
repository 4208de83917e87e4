// Products with 4-bit weights and group scales, many rows (prompts): D = A * W.
//
// The mathematics is that of the row kernel: per group of a weight row the sum of
// a * n runs on the matrix instructions with exact codes, and at the group's end
// s * (sum a*n - z * sum a) joins the fp32 total.  Here the zero point's term is one
// more instruction step of the same sum: with the group's sum of a row of A
// split into three bf16 terms (24 bits together) against -z in three operand
// slots, the accumulator receives - z * sum a.
//
// A workgroup computes BM x 256 of D with waves of 64 x 64 and walks K in chunks of
// 128.  A's chunk is copied straight into one of three LDS stages and read by all
// waves; a wave's codes go from memory to its registers (no other wave of its
// row of waves needs them) one chunk ahead and become operands there.  Per chunk,
// also one chunk ahead, the waves sum A's rows for the zero points.
// 64 x 64 is the wave tile at which neither LDS reads of A (64 bytes per cycle and
// compute unit) nor the conversions (about five vector instructions per
// matrix instruction, of the seven that fit beside it) fill their pipes, and two
// waves fit on a SIMD to cover each other's latencies.
#include "gemm_tiled.h"
#include "w4_operand.h"

namespace mmac {

template <int DT>
__device__ __forceinline__ f32x16 mma32(const i32x4 &a, const i32x4 &b, f32x16 c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// bf16 bits nearest to x, in the low half (finite x of moderate size; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

// WM rows of four waves: BM = 64 * WM.
template <int DT, int QT, int GROUP, int WM>
__global__ __launch_bounds__(WM * 256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_w4_tiled_kernel(W4Params p) {
    constexpr int BM = 64 * WM, BN = kW4Cols, KC = kW4Chunk, NT = WM * 256;
    constexpr int GPC = KC / GROUP, SPG = GROUP / 16;            // groups of a chunk, steps of a group
    constexpr int A_BYTES = BM * KC * 2, STAGES = 3;
    constexpr int EXT_BYTES = GPC * BM * 8;                       // three bf16 terms per row and group
    constexpr int AP = A_BYTES / 16 / NT;                         // copy instructions per chunk
    constexpr int LDS_BYTES = STAGES * A_BYTES + 2 * EXT_BYTES;
    static_assert(LDS_BYTES <= 160 * 1024 / (3 - WM), "LDS: one workgroup of eight waves or two of four per CU");
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    uint8_t *ext = smem + STAGES * A_BYTES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g2 = lane >> 5, l32 = lane & 31, wm = wave >> 2, wn = wave & 3;

    // workgroup -> (tile, range): contiguous runs per XCD, then groups of 8 tile rows column by column
    const int U = p.tiles_m * p.tiles_n * p.split.splits;
    const int x = blockIdx.x & 7, uq = U >> 3, ur = U & 7;
    const int unit = x * uq + (x < ur ? x : ur) + (blockIdx.x >> 3);
    const int tile = unit / p.split.splits, split = unit % p.split.splits;
    const int first = tile / (8 * p.tiles_n) * 8, gsz = min(p.tiles_m - first, 8), in = tile % (8 * p.tiles_n);
    const int row0 = (first + in % gsz) * BM, col0 = in / gsz * BN;

    const int rows = min(p.M - row0, BM), cols = min(p.N - col0, BN);
    const int row_bytes = (p.K + 31) / 32 * 16;
    const rsrc_t ra = make_rsrc(p.A + (int64_t)row0 * p.a_pitch, (uint32_t)(rows * p.a_pitch));
    const rsrc_t rw = make_rsrc(p.codes + (int64_t)col0 * p.pitch, (uint32_t)((cols - 1) * p.pitch + row_bytes));
    const rsrc_t rs = make_rsrc(p.words + col0, (uint32_t)(((p.groups - 1) * p.ldw + cols) * 4));
    const int nall = (p.K + KC - 1) / KC, nfull = p.K / KC;
    const int c0 = split * p.split.per_split, c1 = min(c0 + p.split.per_split, nall);

    // A's chunk c -> LDS rows of 256 bytes, unit u of row r at u ^ (r mod 16)
    const auto copy_a = [&](int c, uint8_t *st) {
        if (c < nfull) {
#pragma unroll
            for (int j = 0; j < AP; ++j) {
                const uint32_t P = j * NT + wave * 64 + lane, r = P >> 4, u = (P & 15) ^ (r & 15);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(st + (j * NT + wave * 64) * 16), 16,
                                                         r * (uint32_t)p.a_pitch + (uint32_t)c * (KC * 2) + u * 16, 0, 0, 0);
            }
        } else {   // K ends inside: through registers, zero past K
            for (int j = 0; j < AP; ++j) {
                const uint32_t P = j * NT + tid, r = P >> 4, u = (P & 15) ^ (r & 15);
                const int e0 = c * KC + (int)u * 8;
                *reinterpret_cast<i32x4 *>(st + P * 16) = masked_unit<2>(ra, r * (uint32_t)p.a_pitch + (uint32_t)e0 * 2, e0, p.K);
            }
        }
    };
    // this lane's codes of chunk c: columns wn * 64 + 32 j + l32, 16-byte units 2 h + g2; and their scale words
    const auto load_w = [&](int c, i32x4 (&cd)[2][2], uint32_t (&sw)[2][GPC]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t col = wn * 64 + j * 32 + l32;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                cd[j][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, col * (uint32_t)p.pitch + (uint32_t)c * (KC / 2) + (2 * h + g2) * 16, 0, 0);
#pragma unroll
            for (int g = 0; g < GPC; ++g) {
                const int gi = p.group == 0 ? 0 : c * GPC + g;
                sw[j][g] = __builtin_amdgcn_raw_buffer_load_b32(
                    rs, gi < p.groups ? (uint32_t)((gi * p.ldw + col) * 4) : kOutOfRange, 0, 0);
            }
        }
    };
    // sums of A's rows over each group of the chunk in `st`, three bf16 terms each: a wave has 16 rows, four
    // lanes (32 elements each) a row
    const auto sum_rows = [&](const uint8_t *st, uint8_t *to) {
        const int r = wave * 16 + (lane >> 2), part = lane & 3;
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const i32x4 v = *reinterpret_cast<const i32x4 *>(st + r * 256 + (((4 * part + u) ^ (r & 15)) << 4));
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int w = v[d];
                if constexpr (DT == DT_BF16)
                    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
                else
                    sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
            }
        }
        const auto add = [](uint32_t a, uint32_t b) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
        };
        uint32_t s = __builtin_bit_cast(uint32_t, sum);
        if constexpr (GROUP >= 64) s = add(s, dpp<kDppXor1>(s));
        if constexpr (GROUP >= 128) s = add(s, dpp<kDppXor2>(s));
        sum = __builtin_bit_cast(float, s);
        const uint32_t hi = bf16_bits(sum);
        const float r1 = sum - __builtin_bit_cast(float, hi << 16);
        const uint32_t mid = bf16_bits(r1), lo = bf16_bits(r1 - __builtin_bit_cast(float, mid << 16));
        if (part % (GROUP / 32) == 0)
            *reinterpret_cast<u32x2 *>(to + (part / (GROUP / 32) * BM + r) * 8) = u32x2{hi | (mid << 16), lo};
    };

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};

    i32x4 cd[2][2];
    uint32_t sw[2][GPC];
    if (c0 < c1) {
        copy_a(c0, smem);
        if (c0 + 1 < c1) copy_a(c0 + 1, smem + A_BYTES);
        load_w(c0, cd, sw);
        wait_vm_lgkm0<0>();
        block_barrier();
        if constexpr (QT == DT_U4) sum_rows(smem, ext);
        wait_vm_lgkm0<0>();
        block_barrier();
    }
    int cur = 0;
    for (int c = c0; c < c1; ++c) {
        const uint8_t *st = smem + cur * A_BYTES;
        const int next = cur == 2 ? 0 : cur + 1, after = next == 2 ? 0 : next + 1;
        const uint8_t *ex = ext + ((c - c0) & 1) * EXT_BYTES;
        if (c + 2 < c1) copy_a(c + 2, smem + after * A_BYTES);
        i32x4 cd1[2][2];
        uint32_t sw1[2][GPC];
        if (c + 1 < c1) {
            load_w(c + 1, cd1, sw1);
            if constexpr (QT == DT_U4) sum_rows(smem + next * A_BYTES, ext + ((c + 1 - c0) & 1) * EXT_BYTES);
        }
        // operand order: GROUP >= 64, step 4 h + d is word d of the lane's unit 2 h + g2; GROUP 32: the lane halves
        // trade words so that every two steps are one unit
        if constexpr (GROUP == 32) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        const auto t = __builtin_amdgcn_permlane32_swap((uint32_t)cd[j][h][d], (uint32_t)cd[j][h][d + 2], false, false);
                        cd[j][h][d] = (int)t[0];
                        cd[j][h][d + 2] = (int)t[1];
                    }
        }
#pragma unroll
        for (int g = 0; g < GPC; ++g) {
            f32x16 t[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) t[i][j] = f32x16{};
#pragma unroll
            for (int s = g * SPG; s < (g + 1) * SPG; ++s) {
                const int u = GROUP == 32 ? 4 * (s / 2) + 2 * g2 + s % 2 : 4 * (2 * (s / 4) + g2) + s % 4;
                i32x4 a[2], b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = wm * 64 + i * 32 + l32;
                    a[i] = *reinterpret_cast<const i32x4 *>(st + r * 256 + ((u ^ (r & 15)) << 4));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) b[j] = operand_of<DT, QT>((uint32_t)cd[j][s / 4][s % 4]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) t[i][j] = mma32<DT>(a[i], b[j], t[i][j]);
            }
            if constexpr (QT == DT_U4) {   // - z * sum a
                i32x4 a[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x2 e = *reinterpret_cast<const u32x2 *>(ex + (g * BM + wm * 64 + i * 32 + l32) * 8);
                    a[i] = i32x4{g2 ? 0 : (int)e[0], g2 ? 0 : (int)e[1], 0, 0};
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int z = (int)bf16_bits(-(float)(sw[j][g] & 0xffu));
                    const i32x4 b = {z | (z << 16), z, 0, 0};
#pragma unroll
                    for (int i = 0; i < 2; ++i) t[i][j] = mma32<DT_BF16>(a[i], b, t[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float s = __builtin_bit_cast(float, sw[j][g] & ~0xffu);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(s, t[i][j][e], acc[i][j][e]);
            }
        }
        wait_vm_lgkm0<0>();
        block_barrier();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) cd[j][h] = cd1[j][h];
#pragma unroll
            for (int g = 0; g < GPC; ++g) sw[j][g] = sw1[j][g];
        }
        cur = next;
    }

    // ranges joined by the last to arrive, in range order (the partials at device scope, see the tiled GEMM)
    if (p.split.splits > 1) {
        constexpr int TILE_BYTES = BM * BN * 4;
        uint8_t *ws = p.split.partials + (int64_t)tile * p.split.splits * TILE_BYTES;
        const rsrc_t mine = make_rsrc(ws + (int64_t)split * TILE_BYTES, TILE_BYTES);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float e0 = acc[i][j][4 * g], e1 = acc[i][j][4 * g + 1], e2 = acc[i][j][4 * g + 2], e3 = acc[i][j][4 * g + 3];
                    const i32x4 v = {__builtin_bit_cast(int, e0), __builtin_bit_cast(int, e1), __builtin_bit_cast(int, e2),
                                     __builtin_bit_cast(int, e3)};
                    __builtin_amdgcn_raw_buffer_store_b128(v, mine, (uint32_t)((((i * 2 + j) * 4 + g) * NT + tid) * 16), 0, kDeviceScope);
                }
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): the partial has reached device scope
        __syncthreads();
        uint32_t *arrived = reinterpret_cast<uint32_t *>(smem);
        if (tid == 0) {
            const uint32_t before = __hip_atomic_fetch_add(p.split.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (before == (uint32_t)p.split.splits - 1)
                __hip_atomic_store(p.split.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *arrived = before;
        }
        __syncthreads();
        if (*arrived != (uint32_t)p.split.splits - 1) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x16 sum = {};
                for (int r = 0; r < p.split.splits; ++r) {
                    const rsrc_t part = make_rsrc(ws + (int64_t)r * TILE_BYTES, TILE_BYTES);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const i32x4 v = __builtin_amdgcn_raw_buffer_load_b128(
                            part, (uint32_t)((((i * 2 + j) * 4 + g) * NT + tid) * 16), 0, kDeviceScope);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int w = v[e];
                            sum[4 * g + e] += __builtin_bit_cast(float, w);
                        }
                    }
                }
                acc[i][j] = sum;
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = wm * 64 + i * 32 + 8 * (e / 4) + 4 * g2 + e % 4, col = wn * 64 + j * 32 + l32;
                if (r < rows && col < cols) store_out(p.out, row0 + r, col0 + col, acc[i][j][e]);
            }
}

template <int DT, int QT, int GROUP>
static hipError_t launch_tiles(const W4Params &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.split.splits));
    if (w4_tile_rows(p.M) == 64) hipLaunchKernelGGL((gemm_w4_tiled_kernel<DT, QT, GROUP, 1>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gemm_w4_tiled_kernel<DT, QT, GROUP, 2>), grid, dim3(512), 0, s, p);
    return hipGetLastError();
}
template <int DT, int QT>
static hipError_t by_group(const W4Params &p, hipStream_t s) {
    switch (p.group) {
    case 32: return launch_tiles<DT, QT, 32>(p, s);
    case 64: return launch_tiles<DT, QT, 64>(p, s);
    case 0:
    case 128: return launch_tiles<DT, QT, 128>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gemm_w4_tiled(int a, int q, const W4Params &p, hipStream_t s) {
    if (a == DT_BF16) return q == DT_FP4 ? by_group<DT_BF16, DT_FP4>(p, s) : by_group<DT_BF16, DT_U4>(p, s);
    if (a == DT_F16) return q == DT_FP4 ? by_group<DT_F16, DT_FP4>(p, s) : by_group<DT_F16, DT_U4>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
