// Block-scaled products grouped by expert in tiles: e4m3 x e4m3.
#include "../grouped_tiles.h"

namespace mmac {
template hipError_t launch_grouped_op<MmaMX<0, 0>>(GroupTile, const GemmParams &, const Groups &, int64_t, hipStream_t);
template hipError_t launch_grouped_op<MmaMXExact<0, 0>>(GroupTile, const GemmParams &, const Groups &, int64_t, hipStream_t);
}  // namespace mmac
