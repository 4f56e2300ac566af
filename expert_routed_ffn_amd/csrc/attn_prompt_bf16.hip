// Attention of new tokens over a bf16 cache.
#include "attn_prompt_bf16.h"

namespace beam {

hipError_t launch_attn_prompt_bf16(const AttnPromptArgs& a, hipStream_t st) { return launch_prompt_d<A_BF16>(a, st); }

}  // namespace beam
