// attend_tile.cu -- many query rows over caches of the heads' type and of E4M3
// codes with one scale (attend_tile.cuh).
#include "attend_tile.cuh"

namespace bevpool {

cudaError_t attend_tile_timeouts(int64_t *count) { return timeouts_here(count); }

cudaError_t launch_attend_tile(const AttnArgs &a, const AttnPlan &pl) {
    return a.cache == kCacheSame ? launch_attend_tile_of<kCacheSame, 1>(a, pl) : launch_attend_tile_of<kCacheE4M3, 1>(a, pl);
}

}  // namespace bevpool
