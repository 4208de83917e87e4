// Products grouped by expert: dispatch on the element types to the instantiations under inst/.
#include "device.h"
#include "grouped.h"

namespace mmac {

// Defined in grouped_tiles.h, instantiated once per type pair under inst/.
template <class Op>
hipError_t launch_grouped_op(GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s);
template <class Op>
hipError_t launch_grouped_wgrad_op(GroupTile t, const GemmParams &p, const Groups &g, hipStream_t s);
// grouped_rows.hip, grouped_mx_rows.hip
hipError_t launch_gemm_grouped_rows(int dt, GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s);
hipError_t launch_gemm_grouped_mx_rows(int a, int b, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s);

template <class Op>
static hipError_t launch_layout(bool trans_b, GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    return trans_b ? launch_grouped_op<Trans<Op, false, true>>(t, p, g, blocks, s) : launch_grouped_op<Op>(t, p, g, blocks, s);
}
hipError_t launch_gemm_grouped(int dt, bool trans_b, GroupTile t, GemmParams p, Groups g, int64_t blocks, hipStream_t s) {
    if (t == GROUP_16 || t == GROUP_32) return trans_b ? hipErrorInvalidValue : launch_gemm_grouped_rows(dt, t, p, g, blocks, s);
    if (dt == DT_BF16) return launch_layout<MmaDense16<DT_BF16>>(trans_b, t, p, g, blocks, s);
    if (dt == DT_F16) return launch_layout<MmaDense16<DT_F16>>(trans_b, t, p, g, blocks, s);
    return hipErrorInvalidValue;
}

hipError_t launch_gemm_grouped_wgrad(int dt, GroupTile t, GemmParams p, Groups g, hipStream_t s) {
    if (dt == DT_BF16) return launch_grouped_wgrad_op<Trans<MmaDense16<DT_BF16>, true, true>>(t, p, g, s);
    if (dt == DT_F16) return launch_grouped_wgrad_op<Trans<MmaDense16<DT_F16>, true, true>>(t, p, g, s);
    return hipErrorInvalidValue;
}

// Op for outputs of 16 bits or fewer, Exact for fp32.
template <class Op, class Exact>
static hipError_t launch_mx(GroupTile t, const GemmParams &p, const Groups &g, int64_t blocks, hipStream_t s) {
    return p.d_type == OUT_ACC ? launch_grouped_op<Exact>(t, p, g, blocks, s) : launch_grouped_op<Op>(t, p, g, blocks, s);
}
hipError_t launch_gemm_grouped_mx(int a, int b, GroupTile t, GemmParams p, Groups g, int64_t blocks, hipStream_t s) {
    if (t == GROUP_16) return launch_gemm_grouped_mx_rows(a, b, p, g, blocks, s);
    // f8f6f4 format selectors: 0 = E4M3, 1 = E5M2
    if (a == DT_E4M3) {
        if (b == DT_E4M3) return launch_mx<MmaMX<0, 0>, MmaMXExact<0, 0>>(t, p, g, blocks, s);
        if (b == DT_E5M2) return launch_mx<MmaMX<0, 1>, MmaMXExact<0, 1>>(t, p, g, blocks, s);
        if (b == DT_FP4) return launch_mx<MmaMX84<0>, MmaMXExact<0, 4>>(t, p, g, blocks, s);
    } else if (a == DT_E5M2) {
        if (b == DT_E4M3) return launch_mx<MmaMX<1, 0>, MmaMXExact<1, 0>>(t, p, g, blocks, s);
        if (b == DT_E5M2) return launch_mx<MmaMX<1, 1>, MmaMXExact<1, 1>>(t, p, g, blocks, s);
        if (b == DT_FP4) return launch_mx<MmaMX84<1>, MmaMXExact<1, 4>>(t, p, g, blocks, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mmac
