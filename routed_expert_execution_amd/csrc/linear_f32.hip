// The 4-bit row products for f32 activations (linear_rows.h).
#include "linear_rows.h"

namespace moe {

hipError_t launch_linear_rows_f32(const LinearArgs& a, bool gated, const DensePlan& p, hipStream_t s) {
    return gated ? linear::launch_rows_t<false, true>(a, p, s) : linear::launch_rows_t<false, false>(a, p, s);
}

}  // namespace moe
