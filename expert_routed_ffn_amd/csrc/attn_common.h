// What the attention kernels share: the cache's 8- and 4-bit elements as bf16.
#pragma once

#include "common.h"
#include "kernels.h"

namespace beam {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// four e4m3 codes to bf16 (exact): codes 0, 1 and codes 2, 3
BEAM_DEV uint32_t e4m3_lo(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
}
BEAM_DEV uint32_t e4m3_hi(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
}

// 2^(b - 127) of an E8M0 byte; 2^-127 is the one that is no normal number
BEAM_DEV float e8m0(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }

// Elements 2 * PAIR and 2 * PAIR + 1 of eight E2M1 codes times their scale, to
// bf16: exact for every code and every scale byte below 255.  Of `scale` the
// conversion takes the exponent field alone, 0 as 2^-127 (all were gone through,
// with other bits set and clear): an E8M0 byte need only be shifted there.
template <int PAIR> BEAM_DEV uint32_t e2m1_pair(uint32_t c, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, PAIR));
}

}  // namespace beam
