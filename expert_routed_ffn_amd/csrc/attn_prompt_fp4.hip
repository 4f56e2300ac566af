// Attention of new tokens over a 4-bit cache.
#include "attn_prompt_bf16.h"

namespace beam {

hipError_t launch_attn_prompt_fp4(const AttnPromptArgs& a, hipStream_t st) { return launch_prompt_d<A_FP4>(a, st); }

}  // namespace beam
