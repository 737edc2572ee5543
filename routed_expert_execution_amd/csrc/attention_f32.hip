// Attention over packed sequences in fp32 (attention_forward.h).
#include "attention_forward.h"

namespace moe {
hipError_t launch_attention_f32(const PackedArgs& a, hipStream_t s) { return packed::launch_forward_by_width<false>(a, s); }
}  // namespace moe
