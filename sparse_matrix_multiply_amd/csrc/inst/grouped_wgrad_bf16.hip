// Weight gradient of products grouped by expert, bf16.
#include "../grouped_tiles.h"

namespace mmac {
template hipError_t launch_grouped_wgrad_op<Trans<MmaDense16<DT_BF16>, true, true>>(GroupTile, const GemmParams &, const Groups &, hipStream_t);
}  // namespace mmac
