// How the attention of new tokens cuts blocks into parts, and its launch.
#include "attn_prompt.h"

namespace beam {

// Parts of the blocks' spans.  Few blocks (together fewer than kWantWG
// workgroups, what the chip holds at once at D <= 128): each may be cut, so that
// the chip has work.  Many: only a sequence that is one block is, where it would
// run on long after the others, into parts of kLongPart at least and kMostWG
// workgroups.  (48 heads over 8 of 128, inputs in the last-level cache, with kWantWG
// 256, 512, 1024: 4 x 8 tokens over 32768 84, 58, 61 us, 128 over 8192 58, 46, 56.  kMostWG 1024, 2048, 4096: 64
// single tokens over 8192 and a chunk of 2048 257, 227, 221, 200 of 2000 and 4
// chunks, e4m3, 120, 119, 143.  kLongPart 512, 1024, 4096: 8 single tokens and 4
// chunks, 4 bits, 65, 62, 95.)
//   A part is kPromptMinPart tokens at least, of what a block sees in the mean:
// among a prompt's own tokens half of them (one prompt of 300 tokens 17.1 us in two
// parts, 12.8 in one; 512: 23.1 and 17.2; but 128 tokens over 500 17.1 in three, 20.1
// in one).  From a quarter of kWantWG on no part is shorter (2 x 256 tokens, window
// 512: 25.6 us in three, 20.2 in one).
//   So among 1024 / Hkv sequences and more a single block is not cut, and a longer
// one among many never: one token behind 131072 among 63, 127, 128 of 500 (8
// key-value heads) takes 583, 1142, 2173 us, where decode, which lists parts by the
// lengths there are, takes 108, 132, 133; 1400 tokens over 32768 are 528 workgroups,
// hence two rounds of uncut ones: 680 TFLOP/s, where 1000 in parts reach 910 and 2048
// 962.
//   With more than half of kWantWG, parts are two or three, and cost a join: none
// where they would be short (one prompt of 700 tokens 30 us in two parts, 22 in
// one; 1300: 56 and 39; but 1000 over 16384: 463 and 505, 8 of up to 128 over
// 8192, e4m3, 74 and 97), and single blocks are cut as among many (40 of up to 8
// tokens over 8192: 121 us with each block cut, 107).
constexpr int kWantWG = 512, kMostWG = 2048, kLongPart = 1024;
// Sequences of this many rows in the mean, or fewer, may be single tokens beside a
// few chunks, whose blocks share their rows between half the waves (64 tokens and 8
// chunks of 2048: 217 us without, 205 with; 16 chunks of 512 the same either way).
constexpr int kFewRows = 2048;
PromptSplit attn_prompt_split(int B, int T, int Hq, int Hkv, int max_len, int window, int sinks) {
    PromptSplit p;
    const int64_t G = Hq / Hkv;
    p.nseq = (uint32_t)B;
    p.blocks = (uint32_t)((int64_t)T * G / kPromptRows + B);
    // what a block's rows see at most: a window, its tokens' breadth and sinks
    int64_t span = max_len;
    if (window > 0) {
        const int64_t seen = (int64_t)window + kPromptRows / G + 32 + (((int64_t)sinks + 15) & ~(int64_t)15);
        span = seen < span ? seen : span;
    }
    const int64_t wg = (int64_t)p.blocks * Hkv;
    const bool half = 2 * wg > kWantWG;
    p.every = wg < kWantWG && !(half && T * G <= (int64_t)kPromptRows / 2 * B);
    p.few = T * G <= (int64_t)kFewRows * B;
    int64_t s, most;
    if (p.every) {
        s = (kWantWG + wg - 1) / wg;
        const int64_t n = T / B, mean = span - (n < span ? n : span) / 2;
        const int64_t up = 4 * wg > kWantWG ? 0 : kPromptMinPart - 1;
        most = half ? span / kLongPart : (mean + up) / kPromptMinPart;
    } else {
        // some sequence may be one block only if there are several
        s = B > 1 ? kMostWG / ((int64_t)B * Hkv) : 1;
        most = (span + kLongPart - 1) / kLongPart;
    }
    s = s < most ? s : most;
    p.S = (uint32_t)(s < 1 ? 1 : s);
    return p;
}

size_t attn_prompt_ws_bytes(int Hkv, int D, const PromptSplit& p) {
    return (size_t)p.slots() * Hkv * kPromptRows * (D + 4) * sizeof(float);
}

hipError_t launch_attn_prompt(AttnPromptArgs a, void* ws, hipStream_t st) {
    a.parts = static_cast<float*>(ws);
    a.ml = reinterpret_cast<float4*>(a.parts + (size_t)a.p.slots() * a.Hkv * kPromptRows * a.D);
    if (a.c.kind == A_F32) return launch_attn_prompt_f32(a, st);
    if (a.c.kind == A_BF16) return launch_attn_prompt_bf16(a, st);
    if (a.c.kind == A_FP8) return launch_attn_prompt_fp8(a, st);
    return launch_attn_prompt_fp4(a, st);
}

}  // namespace beam
