// Products grouped by expert in tiles: f16, weights N x K or (input gradient) read as K x N.
#include "../grouped_tiles.h"

namespace mmac {
template hipError_t launch_grouped_op<MmaDense16<DT_F16>>(GroupTile, const GemmParams &, const Groups &, int64_t, hipStream_t);
template hipError_t launch_grouped_op<Trans<MmaDense16<DT_F16>, false, true>>(GroupTile, const GemmParams &, const Groups &, int64_t, hipStream_t);
}  // namespace mmac
