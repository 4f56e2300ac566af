// Decode with sinks beside the window, over bf16, fp32 and e4m3 caches.
#include "attn_decode.h"

namespace beam {

hipError_t launch_attn_decode_sinks(const AttnDecodeArgs& a, hipStream_t st) {
    if (a.c.kind == A_F32) return launch_decode_d<A_F32, true>(a, st);
    if (a.c.kind == A_BF16) return launch_decode_d<A_BF16, true>(a, st);
    return launch_decode_d<A_FP8, true>(a, st);
}

}  // namespace beam
