// Backward pass of attention over packed sequences in fp32 (attention_backward.h).
#include "attention_backward.h"

namespace moe {
hipError_t launch_attention_backward_f32(const PackedArgs& a, hipStream_t s) { return packed::launch_backward_by_width<false>(a, s); }
}  // namespace moe
