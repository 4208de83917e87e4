// Products grouped by expert for few rows a group (16-bit elements): 16 or 32 rows of one group stream that group's
// weights once, as the skinny GEMM does for a whole product.
//
// HBM bounds it: 2 rows through 2 of 16 experts of 4096 x 4096 bf16, 67 MB, take 15 us (4.5 TB/s; launch and the search for the
// group are 3 of them); 16 rows through 16 such experts 113 us (4.7 TB/s).
#include "grouped.h"
#include "skinny.h"

namespace mmac {

template <class Op, int MB, int NSLOT>
__global__ __launch_bounds__(512) void gemm_grouped_rows_kernel(GemmParams p, Groups q) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[skinny_lds<Op, MB, 1, 8, NSLOT>()];
    GroupTileAt at;
    if (!find_group_tile<16 * MB, HALF_NONE>(q, p.tiles_n, p.group_m, blockIdx.x, at)) return;
    take_group(p, q, at, at.top);
    p.M = min(p.M, 16 * MB);
    skinny_columns<Op, MB, 1, 8, NSLOT>(p, at.tn, smem);
}

template <class Op>
static hipError_t launch_rows(GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    const dim3 grid((unsigned)blocks);
    if (t == GROUP_16) hipLaunchKernelGGL((gemm_grouped_rows_kernel<Op, 1, 4>), grid, dim3(512), 0, s, p, g);
    else hipLaunchKernelGGL((gemm_grouped_rows_kernel<Op, 2, 3>), grid, dim3(512), 0, s, p, g);
    return hipGetLastError();
}

hipError_t launch_gemm_grouped_rows(int dt, GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    if (dt == DT_BF16) return launch_rows<Mma16<DT_BF16, DT_BF16>>(t, p, g, blocks, s);
    if (dt == DT_F16) return launch_rows<Mma16<DT_F16, DT_F16>>(t, p, g, blocks, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
