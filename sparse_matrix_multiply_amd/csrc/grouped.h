// Products grouped by expert (include/mmac_grouped.h): parameters, launchers, and how a workgroup finds its work.
#pragma once

#include "launch.h"

namespace mmac {

// What a grouped product adds to GemmParams, which describe the whole arrays: M rows in all, B and bias of group 0,
// K (the weight gradient: M, N the shape of a group's D; its K is a group's number of rows).
struct Groups {
    const int32_t *offsets;   // count + 1
    int count;
    int rows;                 // rows of the arrays: no offset counts for more
    int64_t b_stride;         // bytes from one group's B to the next
    int64_t sb_stride;        // words, block-scaled B
    int64_t bias_stride;      // fp32 values
    int64_t c_stride, d_stride;   // bytes, weight gradient
    int span;                 // weight gradient: rows that one buffer descriptor may cover, a multiple of the k-tile
};

// Tiles of the grouped kernels: TileShape's, and 16 or 32 rows that stream their group's weights.
enum GroupTile : int { GROUP_16, GROUP_32, GROUP_64, GROUP_128, GROUP_128x256, GROUP_256 };
inline int group_rows(GroupTile t) {
    return t == GROUP_16 ? 16 : t == GROUP_32 ? 32 : t == GROUP_64 ? 64 : t == GROUP_256 ? 256 : 128;
}
inline int group_cols(GroupTile t) {
    return t == GROUP_16 || t == GROUP_32 ? 16 : t == GROUP_64 ? 64 : t == GROUP_128 ? 128 : 256;
}
// Columns of a workgroup of the block-scaled kernels that stream the weights.
constexpr int kMxRowsCols = 32;

hipError_t launch_gemm_grouped(int dt, bool trans_b, GroupTile t, GemmParams p, Groups g, int64_t grid, hipStream_t s);
hipError_t launch_gemm_grouped_wgrad(int dt, GroupTile t, GemmParams p, Groups g, int64_t grid, hipStream_t s);
hipError_t launch_gemm_grouped_mx(int dt_a, int dt_b, GroupTile t, GemmParams p, Groups g, int64_t grid, hipStream_t s);

#if defined(__HIPCC__)

// A workgroup's tile: rows first .. first + rows - 1 of the arrays are group g's, (tm, tn) the tile within them.
struct GroupTileAt {
    int g, first, rows, tm, tn;
};

// Workgroup -> (group, tile), from the offsets alone.  Every wave looks for itself, 64 groups at a time: lane i has group
// base + i, its number of tile rows, and the sum of those before it.  The tiles are numbered group by group,
// within a group as tile_coords numbers them, and dealt to the XCDs in contiguous runs, so tiles that share a
// group's weights are in one L2.  Returns false for the workgroups behind the last tile: the host only
// knows the most tiles there can be.  A range that leaves the arrays is cut to them, a decreasing one is empty.
template <int BM>
__device__ __forceinline__ bool find_group_tile(const Groups &q, int tiles_n, int group_m, int wg, GroupTileAt &at) {
    const int lane = threadIdx.x & 63;
    const auto tiles_of = [&](int g, int &first, int &rows) {
        first = 0;
        int end = 0;
        if (g < q.count) {
            first = min(max(q.offsets[g], 0), q.rows);
            end = min(max(q.offsets[g + 1], first), q.rows);
        }
        rows = end - first;
        return (rows + BM - 1) / BM;
    };
    const auto up_to = [&](int v) {   // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(v, d);
            v += lane >= d ? x : 0;
        }
        return v;
    };
    int first, rows, sum = 0;
    const int own0 = up_to(tiles_of(lane, first, rows));
    int total = __builtin_amdgcn_readlane(own0, 63);
    const int first0 = first, rows0 = rows;
    for (int base = 64; base < q.count; base += 64) total += __builtin_amdgcn_readlane(up_to(tiles_of(base + lane, first, rows)), 63);

    const int U = total * tiles_n, x = wg & 7, local = wg >> 3, per = U >> 3, more = U & 7;
    if (local >= per + (x < more ? 1 : 0)) return false;
    const int u = x * per + min(x, more) + local, row_tile = u / tiles_n;
    int up = own0, base = 0;
    first = first0;
    rows = rows0;
    for (;;) {
        const uint64_t beyond = __ballot(sum + up > row_tile);
        if (beyond) {
            const int l = __builtin_ctzll(beyond);
            at.g = base + l;
            at.first = __builtin_amdgcn_readlane(first, l);
            at.rows = __builtin_amdgcn_readlane(rows, l);
            const int mine = (at.rows + BM - 1) / BM;
            const int in = u - (sum + __builtin_amdgcn_readlane(up, l) - mine) * tiles_n;
            const int per_band = group_m * tiles_n, band = in / per_band, top = band * group_m;
            const int high = min(mine - top, group_m), rest = in - band * per_band;
            at.tm = top + rest % high;
            at.tn = rest / high;
            return true;
        }
        sum += __builtin_amdgcn_readlane(up, 63);
        base += 64;
        if (base >= q.count) return false;   // not reached: row_tile is below the total
        up = up_to(tiles_of(base + lane, first, rows));
    }
}

// The group's part of the arrays (forward and input gradient).
__device__ __forceinline__ void take_group(GemmParams &p, const Groups &q, const GroupTileAt &at) {
    const int es = p.d_type == 0 ? 4 : p.d_type <= 2 ? 2 : 1;
    p.A += (int64_t)at.first * p.a_pitch;
    p.B += at.g * q.b_stride;
    p.D = static_cast<uint8_t *>(p.D) + (int64_t)at.first * p.ldd * es;
    if (p.use_c) p.C = static_cast<const uint8_t *>(p.C) + (int64_t)at.first * p.ldc * es;
    if (p.bias) p.bias += at.g * q.bias_stride;
    p.M = at.rows;
}

#endif  // __HIPCC__

}  // namespace mmac
