// attend_few.cu -- few query rows over caches of the heads' type and of E4M3
// codes with one scale (attend_few.cuh).
#include "attend_few.cuh"

namespace bevpool {

cudaError_t launch_attend_few(const AttnArgs &a, const AttnPlan &pl) {
    return a.cache == kCacheSame ? launch_attend_few_of<kCacheSame>(a, pl) : launch_attend_few_of<kCacheE4M3>(a, pl);
}

}  // namespace bevpool
