// Skinny dense GEMM (M <= 32): dispatch on the element-type pair (the kernel is in skinny.h).
#include "skinny.h"

namespace mmac {

template <class Op, int MB, int CB, int WK, int NSLOT>
__global__ __launch_bounds__(WK * 64) void gemm_skinny_kernel(GemmParams p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[skinny_lds<Op, MB, CB, WK, NSLOT>()];
    skinny_columns<Op, MB, CB, WK, NSLOT>(p, blockIdx.x, smem);
}

template <int DA, int DB>
static hipError_t launch_types(const GemmParams &p, hipStream_t s) {
    typedef Mma16<DA, DB> Op;
    // 8 waves, each with 4 chunks (16 KiB) of copies in flight; 3 chunks (18 KiB) when A has 32 rows
    constexpr int CB = 1, WK = 8;
    const dim3 grid((p.N + 16 * CB - 1) / (16 * CB)), block(WK * 64);
    if (p.M <= 16) hipLaunchKernelGGL((gemm_skinny_kernel<Op, 1, CB, WK, 4>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((gemm_skinny_kernel<Op, 2, CB, WK, 3>), grid, block, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_gemm_skinny(int a, int b, GemmParams p, hipStream_t s) {
    if (p.M > 32) return hipErrorInvalidValue;
    if (a == DT_BF16 && b == DT_BF16) return launch_types<DT_BF16, DT_BF16>(p, s);
    if (a == DT_F16 && b == DT_F16) return launch_types<DT_F16, DT_F16>(p, s);
    if (a == DT_I8 && b == DT_I8) return launch_types<DT_I8, DT_I8>(p, s);
    if (a == DT_E4M3 && b == DT_E4M3) return launch_types<DT_E4M3, DT_E4M3>(p, s);
    if (a == DT_E4M3 && b == DT_E5M2) return launch_types<DT_E4M3, DT_E5M2>(p, s);
    if (a == DT_E5M2 && b == DT_E4M3) return launch_types<DT_E5M2, DT_E4M3>(p, s);
    if (a == DT_E5M2 && b == DT_E5M2) return launch_types<DT_E5M2, DT_E5M2>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
