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
inline int group_threads(GroupTile t) { return t == GROUP_64 || t == GROUP_128 ? 256 : 512; }
// Workgroups of the weight gradient: `per` tiles a group, which share them out to the XCDs where there are some for each.
inline int64_t wgrad_blocks(int64_t per, int64_t groups) { return (per >= 64 ? (per + 7) / 8 * 8 : per) * groups; }
// Columns of a workgroup of the block-scaled kernels that stream the weights.
constexpr int kMxRowsCols = 32;

hipError_t launch_gemm_grouped(int dt, bool trans_b, GroupTile t, GemmParams p, Groups g, int64_t grid, hipStream_t s);
hipError_t launch_gemm_grouped_wgrad(int dt, GroupTile t, GemmParams p, Groups g, hipStream_t s);
hipError_t launch_gemm_grouped_mx(int dt_a, int dt_b, GroupTile t, GemmParams p, Groups g, int64_t grid, hipStream_t s);

#if defined(__HIPCC__)

// A workgroup's tile: rows first .. first + rows - 1 of the arrays are group g's; the tile begins at row `top` of them, in
// column tile tn.  low: the tile is one of BM / 2 rows.
struct GroupTileAt {
    int g, first, rows, top, tn;
    bool low;
};

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int lanes_up_to(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int x = __shfl_up(v, d);
        v += lane >= d ? x : 0;
    }
    return v;
}

// What is left of a group's rows after whole tiles may take a tile of half the rows where it fits one.
//   HALF_IN_PLACE  at its place beside the group's other tiles, with which it shares the weights in the L2.
//   HALF_LAST      after all whole tiles, so that the compute units that are free first at the end find short work; its weights are
//                  read from memory once more.
// Measured (bf16, lognormal groups, us in place / last): 256 rows, 20 groups of 300 x 2048 x 4096 166 / 144, 16 of 512 x 4096 x 2048 212
// / 202, 16 of 1024 x 4096 x 2048 303 / 300; 128 rows, 16 of 256 x 4096 x 4096 213 / 222, 32 of 256 x 2048 x 4096 214 / 233.
enum : int { HALF_NONE, HALF_IN_PLACE, HALF_LAST };

// Workgroup -> (group, tile), from the offsets alone.  Every wave looks for itself, 64 * PER groups at a time: a lane has PER
// neighbouring ones (their offsets are loaded together), their tile rows, and the sum of those before it.  Four a lane for more
// than 64 groups (8 rows through 256 experts of 2048^2: 22 us, 28 with 64 groups at a time), one up to 64 (16 rows through 64 experts
// in 4 bits: 32.2 us, 33.9 with four).  Tiles are BM rows high; whole ones and those of HALF_LAST
// are numbered each group by group, within a group in bands of group_m tile rows, column by column, and dealt to the
// XCDs in contiguous runs, so tiles that share a group's weights run at about the same time on one L2.  Returns false
// for the workgroups behind the last tile: the host only knows the most tiles there can be.  A range that leaves
// the arrays is cut to them, a decreasing one is empty.
template <int BM, int HALF, int PER>
__device__ __forceinline__ bool find_group_tile_by(const Groups &q, int tiles_n, int group_m, int wg, GroupTileAt &at) {
    const int lane = threadIdx.x & 63;
    const auto whole = [](int rows) { return (rows + (HALF == HALF_LAST ? BM / 2 : BM) - 1) / BM; };
    const auto half = [](int rows) { return rows % BM > 0 && rows % BM <= BM / 2 ? 1 : 0; };
    // the lane's groups of the 64 * PER from `base` on; those behind the last one have no rows
    const auto load = [&](int base, int (&first)[PER], int (&rows)[PER]) {
        int o[PER + 1];
#pragma unroll
        for (int j = 0; j <= PER; ++j) o[j] = q.offsets[min(base + lane * PER + j, q.count)];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            first[j] = min(max(o[j], 0), q.rows);
            rows[j] = min(max(o[j + 1], first[j]), q.rows) - first[j];   // cut before it is subtracted: any 32-bit value may come
        }
    };
    const auto sum_of = [&](const int (&rows)[PER], bool low) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) n += low ? half(rows[j]) : whole(rows[j]);
        return n;
    };
    int first[PER], rows[PER];
    int total = 0, total_low = 0, up = 0, up_low = 0;
    for (int base = 0; base < q.count; base += 64 * PER) {
        load(base, first, rows);
        total += __builtin_amdgcn_readlane(up = lanes_up_to(sum_of(rows, false)), 63);
        if (HALF == HALF_LAST) total_low += __builtin_amdgcn_readlane(up_low = lanes_up_to(sum_of(rows, true)), 63);
    }
    const int x = wg & 7;
    int local = wg >> 3, U = total * tiles_n, mine = (U >> 3) + (x < (U & 7) ? 1 : 0);
    at.low = false;
    if (HALF == HALF_LAST && local >= mine) {
        local -= mine;
        U = total_low * tiles_n;
        mine = (U >> 3) + (x < (U & 7) ? 1 : 0);
        at.low = true;
    }
    if (local >= mine) return false;
    const int u = x * (U >> 3) + min(x, U & 7) + local, row_tile = u / tiles_n;
    int before = 0;   // tile rows of the groups before
    for (int base = 0; base < q.count; base += 64 * PER) {
        if (q.count > 64 * PER) {   // else they are still there
            load(base, first, rows);
            up = lanes_up_to(sum_of(rows, at.low));
        } else if (at.low) {
            up = up_low;
        }
        const uint64_t beyond = __ballot(before + up > row_tile);
        if (!beyond) {
            before += __builtin_amdgcn_readlane(up, 63);
            continue;
        }
        const int l = __builtin_ctzll(beyond);
        before += l > 0 ? __builtin_amdgcn_readlane(up, l - 1) : 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int r = __builtin_amdgcn_readlane(rows[j], l), count = at.low ? half(r) : whole(r);
            if (row_tile >= before + count) {
                before += count;
                continue;
            }
            const int in = u - before * tiles_n, per_band = group_m * tiles_n, band = in / per_band, above = band * group_m;
            const int high = min(count - above, group_m), rest = in - band * per_band;
            at.g = __builtin_amdgcn_readfirstlane(base + l * PER + j);
            at.first = __builtin_amdgcn_readlane(first[j], l);
            at.rows = r;
            at.top = __builtin_amdgcn_readfirstlane(at.low ? r / BM * BM : (above + rest % high) * BM);
            at.tn = __builtin_amdgcn_readfirstlane(rest / high);
            if (HALF == HALF_IN_PLACE) at.low = r - at.top <= BM / 2;
            // holds but for offsets so wrong that the sums above passed 31 bits
            return at.g < q.count && (uint32_t)at.top < (uint32_t)r && (uint32_t)at.tn < (uint32_t)tiles_n;
        }
        return false;   // not reached: the lane's tiles pass row_tile
    }
    return false;       // not reached: row_tile is below the total
}
template <int BM, int HALF>
__device__ __forceinline__ bool find_group_tile(const Groups &q, int tiles_n, int group_m, int wg, GroupTileAt &at) {
    return q.count <= 64 ? find_group_tile_by<BM, HALF, 1>(q, tiles_n, group_m, wg, at)
                         : find_group_tile_by<BM, HALF, 4>(q, tiles_n, group_m, wg, at);
}

// The group's part of the arrays (forward and input gradient), from row `from` of its rows on.
__device__ __forceinline__ void take_group(GemmParams &p, const Groups &q, const GroupTileAt &at, int from) {
    const int es = p.d_type == 0 ? 4 : p.d_type <= 2 ? 2 : 1;
    const int64_t row = at.first + from;
    p.A += row * p.a_pitch;
    p.B += at.g * q.b_stride;
    p.D = static_cast<uint8_t *>(p.D) + row * p.ldd * es;
    if (p.use_c) p.C = static_cast<const uint8_t *>(p.C) + row * p.ldc * es;
    if (p.bias) p.bias += at.g * q.bias_stride;
    p.M = at.rows - from;
}

#endif  // __HIPCC__

}  // namespace mmac
