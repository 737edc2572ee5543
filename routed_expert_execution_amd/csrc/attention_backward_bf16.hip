// Backward pass of attention over packed sequences in bf16 (attention_backward.h).
#include "attention_backward.h"

namespace moe {
hipError_t launch_attention_backward_bf16(const PackedArgs& a, hipStream_t s) { return packed::launch_backward_by_width<true>(a, s); }
}  // namespace moe
