// How decode cuts sequences into parts, and its launches over bf16, fp32 and e4m3
// caches without sinks.
#include "attn_decode.h"

namespace beam {

AttnSplit attn_decode_split(int B, int Hkv, int max_len, int window, int sinks) {
    // a window's tokens begin inside a 16-token block, and its sinks end in one;
    // together no more than there are (64 sequences of 1000 tokens in windows of 512
    // with 100000 sinks: 40.8 us without a workspace, as without a window; counted
    // whole, 47.1 us with listed parts in 14.4 MB)
    int64_t span = window > 0 && window < max_len ? (int64_t)window + 15 : max_len;
    if (window > 0 && window < max_len && sinks > 0) {
        span += ((int64_t)sinks + 15) & ~(int64_t)15;
        span = span < max_len ? span : max_len;
    }
    const int64_t heads = (int64_t)B * Hkv;
    const auto at_least_1 = [](int64_t v) { return v < 1 ? 1 : v; };
    const auto parts = [&](int of) { return at_least_1((span + of - 1) / of); };
    const int64_t w = at_least_1(kWantWG / heads), cap = at_least_1(kMostWG / heads);
    const int64_t most = w > parts(kMaxPart) ? w : parts(kMaxPart);
    const int64_t s = parts(kMinPart) < most ? parts(kMinPart) : most;
    AttnSplit p;
    p.want = (uint32_t)w;
    p.S = (uint32_t)(s < cap ? s : cap);
    p.extra = cap < parts(kMaxPart) && B > 1 && B < kMostListed ? (uint32_t)at_least_1(kMostWG / Hkv) : 0;
    p.rows = p.extra ? (uint64_t)B * p.want + p.extra : (uint64_t)B * p.S;
    p.joins = p.extra && p.rows - B < (uint64_t)B ? (uint32_t)(p.rows - B) : (uint32_t)B;
    return p;
}

size_t attn_decode_ws_bytes(int B, int Hq, int D, const AttnSplit& p) {
    if (p.extra) return (p.rows + p.joins) * sizeof(int4) + p.rows * Hq * (D + 2) * sizeof(float);
    return p.S > 1 ? p.rows * Hq * (D + 2) * sizeof(float) : 0;
}

hipError_t launch_attn_decode(AttnDecodeArgs a, void* ws, hipStream_t st) {
    a.parts = static_cast<float*>(ws);
    if (a.p.extra) {
        a.items = static_cast<int4*>(ws);
        a.lists = a.items + a.p.rows;
        a.parts = reinterpret_cast<float*>(a.lists + a.p.joins);
    }
    if (a.c.kind == A_FP4) return launch_attn_decode_fp4(a, st);
    if (a.sinks > 0) return launch_attn_decode_sinks(a, st);
    if (a.c.kind == A_F32) return launch_decode_d<A_F32, false>(a, st);
    if (a.c.kind == A_BF16) return launch_decode_d<A_BF16, false>(a, st);
    return launch_decode_d<A_FP8, false>(a, st);
}

}  // namespace beam
