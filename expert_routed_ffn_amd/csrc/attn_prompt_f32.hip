// Attention of new tokens over an fp32 cache.
#include "attn_prompt.h"

namespace beam {

hipError_t launch_attn_prompt_f32(const AttnPromptArgs& a, hipStream_t st) { return launch_prompt_d<A_F32>(a, st); }

}  // namespace beam
