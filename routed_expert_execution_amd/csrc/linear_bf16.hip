// The 4-bit row products for bf16 activations (linear_rows.h).
#include "linear_rows.h"

namespace moe {

hipError_t launch_linear_rows_bf16(const LinearArgs& a, bool gated, const DensePlan& p, hipStream_t s) {
    return gated ? linear::launch_rows_t<true, true>(a, p, s) : linear::launch_rows_t<true, false>(a, p, s);
}

}  // namespace moe
