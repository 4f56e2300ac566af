// Attention of new tokens over an e4m3 cache.
#include "attn_prompt_bf16.h"

namespace beam {

hipError_t launch_attn_prompt_fp8(const AttnPromptArgs& a, hipStream_t st) { return launch_prompt_d<A_FP8>(a, st); }

}  // namespace beam
