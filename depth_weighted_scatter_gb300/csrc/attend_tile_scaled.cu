// attend_tile_scaled.cu -- many query rows over E4M3 codes with a scale for each
// page and key head (attend_tile.cuh).
#include "attend_tile.cuh"

namespace bevpool {

cudaError_t attend_tile_scaled_timeouts(int64_t *count) { return timeouts_here(count); }

cudaError_t launch_attend_tile_scaled(const AttnArgs &a, const AttnPlan &pl) { return launch_attend_tile_of<kCacheScaled>(a, pl); }

}  // namespace bevpool
