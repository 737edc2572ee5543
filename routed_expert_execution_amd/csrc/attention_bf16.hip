// Attention over packed sequences in bf16 (attention_forward.h).
#include "attention_forward.h"

namespace moe {
hipError_t launch_attention_bf16(const PackedArgs& a, hipStream_t s) { return packed::launch_forward_by_width<true>(a, s); }
}  // namespace moe
