// attend_tile_scaled_8.cu -- many query rows over E4M3 codes with a scale for each
// page and key head, pages of 16 and 32 slots (attend_tile.cuh).
#include "attend_tile.cuh"

namespace bevpool {

cudaError_t attend_tile_scaled_8_timeouts(int64_t *count) { return timeouts_here(count); }

cudaError_t launch_attend_tile_scaled_8(const AttnArgs &a, const AttnPlan &pl) { return launch_attend_tile_of<kCacheScaled, 8>(a, pl); }

}  // namespace bevpool
