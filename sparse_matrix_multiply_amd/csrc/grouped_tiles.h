// Grouped products in tiles: the tiled kernel's main loop and epilogue on one group's part of the arrays.
//
// Each tile is the dense kernel's, so what bounds it is the same (matrix instructions and the copies that feed them); what is the
// groups' own is the tiles that their last rows leave partly empty, the rounds of tiles, and weights that only two or three
// tile rows share.  8192 rows, 4096 x 4096 bf16: one or two groups 225 to 230 us (1200 TFLOP/s), 16 equal ones 256, 16 of
// lognormal sizes 324 to 331.
#pragma once

#include "gemm_tiled.h"
#include "grouped.h"

namespace mmac {

template <class T, class Op, int BM>
__device__ __forceinline__ void group_tile(const GemmParams &p, const GroupTileAt &at, uint8_t *smem) {
    T t(p, at.top / BM, at.tn, 0, at.first);
    if constexpr (T::SPARE_BYTES > 0) t.spare = smem + T::STAGES * T::STAGE + t.wave * 256;
    walk_k<T, Op>(t, smem);
    t.epilogue(smem);
}

// One workgroup per tile of BM x BN, WM x WN waves, or (HALF) of BM / 2 x BN; PER_CU of them a compute unit.
template <class Op, int BM, int BN, int WM, int WN, int STAGES, int HALF, int PER_CU = 1>
__global__ __launch_bounds__(WM *WN * 64) __attribute__((amdgpu_waves_per_eu(WM * WN * PER_CU / 4, WM * WN * PER_CU / 4)))
void gemm_grouped_kernel(GemmParams p, Groups q) {
    typedef TiledGemm<Op, BM, BN, WM, WN, STAGES> T;
    typedef TiledGemm<Op, HALF ? BM / 2 : BM, BN, WM, WN, HALF ? 3 : STAGES> L;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::LDS_BYTES > L::LDS_BYTES ? T::LDS_BYTES : L::LDS_BYTES];
    GroupTileAt at;
    if (!find_group_tile<BM, HALF>(q, p.tiles_n, p.group_m, blockIdx.x, at)) return;
    take_group(p, q, at, 0);
    if constexpr (T::SCALED) p.sb += at.g * q.sb_stride;
    if constexpr (HALF)
        if (at.low) return group_tile<L, Op, BM / 2>(p, at, smem);
    group_tile<T, Op, BM>(p, at, smem);
}

// The group with the n-th most rows, the lower number first among equals (up to 64 groups, a lane each).
__device__ __forceinline__ int nth_longest(const Groups &q, int n) {
    const int lane = threadIdx.x & 63;
    int rows = -1;
    if (lane < q.count) {
        const int first = min(max(q.offsets[lane], 0), q.rows);
        rows = min(max(q.offsets[lane + 1], first), q.rows) - first;
    }
    int rank = 0;
    for (int j = 0; j < q.count; ++j) {
        const int other = __builtin_amdgcn_readlane(rows, j);
        rank += other > rows || (other == rows && j < lane) ? 1 : 0;
    }
    return __builtin_ctzll(__ballot(rank == n && lane < q.count));
}

// Weight gradient: the tiles of every group's D, the sum over the group's rows (both operands' K is strided).  A sum
// over more rows than one buffer descriptor covers is walked in parts, each with descriptors of its own.
template <class Op, int BM, int BN, int WM, int WN, int STAGES, int PER_CU = 1>
__global__ __launch_bounds__(WM *WN * 64) __attribute__((amdgpu_waves_per_eu(WM * WN * PER_CU / 4, WM * WN * PER_CU / 4)))
void gemm_grouped_wgrad_kernel(GemmParams p, Groups q) {
    typedef TiledGemm<Op, BM, BN, WM, WN, STAGES> T;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::LDS_BYTES];
    // The groups one after the other, a group's tiles in contiguous runs per XCD where there are some for each, so that a long
    // group is every XCD's.  Large tiles of a few groups: the longest group first, so that the short ones fill the end (8 groups of
    // 4096 x 2048 from 8192 rows: 240 us without, 233 with; ranking 49 groups for 64 x 64 tiles takes longer than their work: 178 us
    // without, 230 with).
    const int per = p.tiles_m * p.tiles_n, x = blockIdx.x & 7, share = (per + 7) / 8;
    int g, in;
    if (per >= 64) {
        const int local = blockIdx.x >> 3, mine = local % share;
        g = local / share;
        if (mine >= (per >> 3) + (x < (per & 7) ? 1 : 0)) return;
        in = x * (per >> 3) + min(x, per & 7) + mine;
    } else {
        g = blockIdx.x / per;
        in = blockIdx.x - g * per;
    }
    if (BM == 256 && q.count > 1 && q.count <= 16) g = nth_longest(q, g);
    const int band = in / (p.group_m * p.tiles_n), top = band * p.group_m, high = min(p.tiles_m - top, p.group_m);
    const int rest = in - band * p.group_m * p.tiles_n;
    const int first = __builtin_amdgcn_readfirstlane(min(max(q.offsets[g], 0), q.rows));
    const int end = __builtin_amdgcn_readfirstlane(min(max(q.offsets[g + 1], first), q.rows));
    p.A += (int64_t)first * p.a_pitch;
    p.B += (int64_t)first * p.b_pitch;
    p.D = static_cast<uint8_t *>(p.D) + g * q.d_stride;
    if (p.use_c) p.C = static_cast<const uint8_t *>(p.C) + g * q.c_stride;
    int left = end - first;
    p.K = min(left, q.span);
    T t(p, top + rest % high, rest / high, 0);
    walk_k<T, Op>(t, smem);
    while ((left -= p.K) > 0) {
        block_barrier();   // every wave is done with the stages
        p.A += (int64_t)p.K * p.a_pitch;
        p.B += (int64_t)p.K * p.b_pitch;
        p.K = min(left, q.span);
        t.set_operands();
        walk_k<T, Op>(t, smem, false);
    }
    t.epilogue(smem);
}

template <class Op>
hipError_t launch_grouped_op(GroupTile tile, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    const dim3 grid((unsigned)blocks);
    // workgroups of the small tiles that fit a compute unit's 160 KiB of LDS.  Three of 128 x 128 (FP4 weights) leave 168 registers a
    // wave, 25 too few (22 in the fp32 form), which are spilled and reloaded in the loop of the last k-tiles, not in the steady one; two,
    // without spills, are as fast within noise (us, three / two: 4 x 2048 x 4096^2 128 / 135; 16 x 256 x 4096 x 8192 171 / 167, fp32 231 / 236)
    constexpr int L64 = TiledGemm<Op, 64, 64, 2, 2, 2>::LDS_BYTES, L128 = TiledGemm<Op, 128, 128, 2, 2, 2>::LDS_BYTES;
    constexpr int P64 = 160 * 1024 / L64 < 4 ? 160 * 1024 / L64 : 4, P128 = 160 * 1024 / L128 < 3 ? 160 * 1024 / L128 : 3;
    switch (tile) {
    case GROUP_64: hipLaunchKernelGGL((gemm_grouped_kernel<Op, 64, 64, 2, 2, 2, HALF_NONE, P64>), grid, dim3(256), 0, s, p, g); break;
    case GROUP_128: hipLaunchKernelGGL((gemm_grouped_kernel<Op, 128, 128, 2, 2, 2, HALF_NONE, P128>), grid, dim3(256), 0, s, p, g); break;
    // block-scaled products take this tile for groups of up to 128 rows: a half tile would change little
    case GROUP_128x256: hipLaunchKernelGGL((gemm_grouped_kernel<Op, 128, 256, 2, 4, 3, Op::kScaled ? HALF_NONE : HALF_IN_PLACE>), grid, dim3(512), 0, s, p, g); break;
    case GROUP_256:
        if constexpr (Op::kScaled) return hipErrorInvalidValue;   // no registers left for the scale words
        else hipLaunchKernelGGL((gemm_grouped_kernel<Op, 256, 256, 2, 4, 2, HALF_LAST>), grid, dim3(512), 0, s, p, g);
        break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <class Op>
hipError_t launch_grouped_wgrad_op(GroupTile tile, const GemmParams &p, const Groups &g, hipStream_t s) {
    const dim3 grid((unsigned)wgrad_blocks((int64_t)p.tiles_m * p.tiles_n, g.count));   // as the kernel counts
    switch (tile) {
    case GROUP_64: hipLaunchKernelGGL((gemm_grouped_wgrad_kernel<Op, 64, 64, 2, 2, 2, 5>), grid, dim3(256), 0, s, p, g); break;
    case GROUP_128: hipLaunchKernelGGL((gemm_grouped_wgrad_kernel<Op, 128, 128, 2, 2, 2, 2>), grid, dim3(256), 0, s, p, g); break;
    case GROUP_128x256: hipLaunchKernelGGL((gemm_grouped_wgrad_kernel<Op, 128, 256, 2, 4, 3>), grid, dim3(512), 0, s, p, g); break;
    case GROUP_256: hipLaunchKernelGGL((gemm_grouped_wgrad_kernel<Op, 256, 256, 2, 4, 2>), grid, dim3(512), 0, s, p, g); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace mmac
