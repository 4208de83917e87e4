// Block-scaled products grouped by expert for few rows a group: 16 rows of one group against 32 of its columns, the
// weights streamed once.
//
// 2 * rows flops per element of B are far below the chip's flop/byte ridge, so the time is set by reading B.
// The eight waves of a workgroup split K into contiguous ranges of chunks, 128 bytes of a row of B each (128 8-bit or 256
// 4-bit elements: one or two steps of v_mfma_scale_f32_16x16x128_f8f6f4).  A wave copies its chunk of B and of its scale words
// straight into a private ring of two LDS slots, whole lines at a time, and reads fragments back (a wave reads only what it
// copied: no barrier); two workgroups fit a compute unit, so one streams while the other starts or ends.  The waves' partial tiles are added up in LDS in wave order.
//
// Within a step of 128 elements lane quarter q = lane / 16 holds, of its row (lane mod 16): 8-bit elements
// 16q .. 16q + 15 and 64 + 16q .. 64 + 16q + 15, 4-bit elements 32q .. 32q + 31; its scale operand's byte 0 is the exponent of
// elements 32q .. 32q + 31 in either format.  Established on gfx950 by the products' agreement with the 64-bit sums, every block's
// exponent and every element different; the parity tests recheck it.
//
// Measured: 16 rows through 16 experts of 4096 x 4096 FP4 (143 MB) in 31.7 us (4.5 TB/s).  With A and its scale words in the ring too,
// so that one workgroup filled a compute unit's LDS, 42 us: at K 4096 a wave's range is its two slots, and nothing ran
// while a workgroup started or ended.
#include "grouped.h"
#include "skinny.h"

namespace mmac {

template <int FB> struct MxRows {
    static constexpr int kSteps = FB == 4 ? 2 : 1;          // instruction steps of a chunk
    static constexpr int kElems = 128 * kSteps;
    static constexpr int kB = kMxRowsCols * 128;
    static constexpr int kSlot = kB + 256;                  // B, then its scale words
    static constexpr int kLoads = kB / 1024 + 1 + 3 * kSteps;   // copies and loads of a chunk
    static constexpr int kWaves = 8, kSlots = 2;
    static constexpr int kLds = kWaves * kSlots * kSlot;
    static_assert(kLds >= kWaves * 2 * 4 * 64 * 4, "ring and partial tiles");
};

// EXACT (fp32 outputs): products of bf16 elements instead (see ExactBf16); a lane then holds elements 32q .. 32q + 31 of either
// operand.
template <int FA, int FB, bool EXACT>
__global__ __launch_bounds__(512) void gemm_grouped_mx_rows_kernel(GemmParams p, Groups q) {
    typedef MxRows<FB> R;
    __shared__ __attribute__((aligned(16))) uint8_t smem[R::kLds];
    GroupTileAt at;
    if (!find_group_tile<16, HALF_NONE>(q, p.tiles_n, p.group_m, blockIdx.x, at)) return;
    take_group(p, q, at, at.top);
    p.M = min(p.M, 16);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, quarter = lane >> 4;
    const int col0 = at.tn * kMxRowsCols, cols = min(kMxRowsCols, p.N - col0);
    const int words = p.scale_rows, b_end = FB == 4 ? p.K / 2 : p.K;   // bytes of a row
    const rsrc_t ra = make_rsrc(p.A, (uint32_t)(p.M * p.a_pitch));
    const rsrc_t rb = make_rsrc(p.B + (int64_t)col0 * p.b_pitch, (uint32_t)(cols * p.b_pitch));
    // scale words to the last strip's last one of these rows and columns: the arrays may end there
    const auto strips_of = [&](const uint32_t *w, int64_t ld, int n) { return make_rsrc(w, words > 0 ? (uint32_t)(((words - 1) * ld + n) * 4) : 0u); };
    const rsrc_t rsa = strips_of(p.sa + at.first + at.top, p.ldsa, p.M), rsb = strips_of(p.sb + at.g * q.sb_stride + col0, p.ldsb, cols);
    SkinnyOut<float, 1, 2, R::kWaves> out(p, col0);

    f32x4 acc[1][2] = {};
    const int chunks = (p.K + R::kElems - 1) / R::kElems, per = (chunks + R::kWaves - 1) / R::kWaves;
    const int c0 = min(wave * per, chunks), c1 = min(c0 + per, chunks);
    uint8_t *ring = smem + wave * R::kSlots * R::kSlot;

    // Chunk c: copies of B, 8 rows x 128 bytes an instruction (lane l: row l / 8, unit l mod 8, swizzled as skinny_swz
    // says), and of its scale words, 4 bytes a lane; A's fragments and scale words straight into registers (few
    // rows: what is past them reads as zero without an access).  What lies past K reads as zero.
    i32x4 a[R::kSlots][R::kSteps][2];
    uint32_t wa[R::kSlots][R::kSteps];
    const auto issue = [&](int c, int slot) {
        uint8_t *dst = ring + slot * R::kSlot;
        const int r = lane >> 3;
#pragma unroll
        for (int j = 0; j < R::kB / 1024; ++j) {
            const int row = 8 * j + r;
            const int at_byte = c * 128 + ((lane & 7) ^ skinny_swz(row & 15)) * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(dst + j * 1024), 16,
                                                     at_byte < b_end ? (uint32_t)row * (uint32_t)p.b_pitch + at_byte : kOutOfRange, 0, 0, 0);
        }
        const int tb = c * R::kSteps + (lane >> 5);   // word lane / 32 of column lane mod 32
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsb, (lds_void *)(dst + R::kB), 4,
            (lane >> 5) < R::kSteps && tb < words ? (uint32_t)((tb * p.ldsb + (lane & 31)) * 4) : kOutOfRange, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < R::kSteps; ++v) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at_byte = c * R::kElems + v * 128 + 16 * (EXACT ? 2 * quarter + h : quarter + 4 * h);
                a[slot][v][h] = __builtin_amdgcn_raw_buffer_load_b128(
                    ra, at_byte < p.K ? (uint32_t)r16 * (uint32_t)p.a_pitch + at_byte : kOutOfRange, 0, 0);
            }
            const int ta = c * R::kSteps + v;
            wa[slot][v] = __builtin_amdgcn_raw_buffer_load_b32(rsa, ta < words ? (uint32_t)((ta * p.ldsa + r16) * 4) : kOutOfRange, 0, 0);
        }
        // every load of the chunk is issued here: the counted waits below rely on it
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto unit_at = [&](const uint8_t *block, int u) -> i32x4 {
        return *reinterpret_cast<const i32x4 *>(block + r16 * 128 + ((u ^ skinny_swz(r16)) << 4));
    };

#pragma unroll
    for (int i = 0; i < R::kSlots; ++i)
        if (c0 + i < c1) issue(c0 + i, i);
    for (int first = c0; first < c1; first += R::kSlots) {
#pragma unroll
        for (int slot = 0; slot < R::kSlots; ++slot) {   // registers are indexed by constants
            const int c = first + slot;
            if (c >= c1) break;
            skinny_wait_n<R::kLoads, R::kSlots - 1>(min(R::kSlots - 1, c1 - 1 - c));
            const uint8_t *src = ring + slot * R::kSlot;
            const uint32_t *sb = reinterpret_cast<const uint32_t *>(src + R::kB);
            i32x8 x[R::kSteps], b[R::kSteps][2];
            uint32_t ea[R::kSteps], eb[R::kSteps][2];
#pragma unroll
            for (int v = 0; v < R::kSteps; ++v) {
                const i32x4 lo = a[slot][v][0], hi = a[slot][v][1];
                x[v] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                ea[v] = wa[slot][v];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (FB == 4) {
                        const i32x4 y = unit_at(src + j * 2048, 4 * v + quarter);
                        b[v][j] = i32x8{y[0], y[1], y[2], y[3], 0, 0, 0, 0};
                    } else {
                        const i32x4 y = unit_at(src + j * 2048, EXACT ? 2 * quarter : quarter),
                                    z = unit_at(src + j * 2048, EXACT ? 2 * quarter + 1 : 4 + quarter);
                        b[v][j] = i32x8{y[0], y[1], y[2], y[3], z[0], z[1], z[2], z[3]};
                    }
                    eb[v][j] = sb[v * 32 + j * 16 + r16];
                }
            }
            skinny_wait_lds();   // the slot's reads are done before new data is copied into it
            if (c + R::kSlots < c1) issue(c + R::kSlots, slot);
#pragma unroll
            for (int v = 0; v < R::kSteps; ++v) {
                // blocks at and past K: zeros, whose scale words may hold anything
                const bool in = c * R::kElems + v * 128 + 32 * quarter < p.K;
                const uint32_t sa = in ? ea[v] >> (8 * quarter) : 127u;
                i32x4 xs[4];
                if constexpr (EXACT) ExactBf16<FA>::convert(xs, x[v], sa);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t sc = in ? eb[v][j] >> (8 * quarter) : 127u;
                    if constexpr (EXACT) {
                        i32x4 ys[4];
                        ExactBf16<FB>::convert(ys, b[v][j], sc);
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            acc[0][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xs[n]),
                                                                                __builtin_bit_cast(bf16x8, ys[n]), acc[0][j], 0, 0, 0);
                    } else {
                        acc[0][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x[v], b[v][j], acc[0][j], FA, FB, 0, (int)sa, 0, (int)sc);
                    }
                }
            }
        }
    }
    out.finish(acc, smem);
}

template <int FA, int FB>
static hipError_t launch_as(const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    const dim3 grid((unsigned)blocks);
    if (p.d_type == OUT_ACC) hipLaunchKernelGGL((gemm_grouped_mx_rows_kernel<FA, FB, true>), grid, dim3(512), 0, s, p, g);
    else hipLaunchKernelGGL((gemm_grouped_mx_rows_kernel<FA, FB, false>), grid, dim3(512), 0, s, p, g);
    return hipGetLastError();
}

hipError_t launch_gemm_grouped_mx_rows(int a, int b, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    // f8f6f4 format selectors: 0 = E4M3, 1 = E5M2, 4 = FP4
    if (a == DT_E4M3) {
        if (b == DT_E4M3) return launch_as<0, 0>(p, g, blocks, s);
        if (b == DT_E5M2) return launch_as<0, 1>(p, g, blocks, s);
        if (b == DT_FP4) return launch_as<0, 4>(p, g, blocks, s);
    } else if (a == DT_E5M2) {
        if (b == DT_E4M3) return launch_as<1, 0>(p, g, blocks, s);
        if (b == DT_E5M2) return launch_as<1, 1>(p, g, blocks, s);
        if (b == DT_FP4) return launch_as<1, 4>(p, g, blocks, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mmac
