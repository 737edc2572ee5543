// Attention over a paged cache held in 4 bits, queries in fp32 (in a file of its
// own so that the variants compile side by side).
#include "attention_cached.h"

namespace moe {

hipError_t launch_cached_f32(const CachedArgs& a, const CachedPlan& p, hipStream_t s) { return cached::launch_by_width<false>(a, p, s); }

}  // namespace moe
