// Decode over a 4-bit cache, with sinks or without.
#include "attn_decode.h"

namespace beam {

hipError_t launch_attn_decode_fp4(const AttnDecodeArgs& a, hipStream_t st) {
    return launch_decode_d<A_FP4, true>(a, st);
}

}  // namespace beam
