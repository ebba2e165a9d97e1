// attend_few_scaled.cu -- few query rows over E4M3 codes with a scale for each
// page and key head (attend_few.cuh).
#include "attend_few.cuh"

namespace bevpool {

cudaError_t launch_attend_few_scaled(const AttnArgs &a, const AttnPlan &pl) { return launch_attend_few_of<kCacheScaled>(a, pl); }

}  // namespace bevpool
