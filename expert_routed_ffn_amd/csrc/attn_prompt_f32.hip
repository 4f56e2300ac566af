// Attention of new tokens over an fp32 cache: both products on the fp32 matrix
// instructions, which bound it (one prompt of 4096 tokens, 48 heads over 8 of 128:
// 114 TFLOP/s of the 154 that a large fp32 product reaches; 2048: 118).  Blocks of up
// to 64 rows leave two of the four waves idle: 4 x 8 tokens over up to 32768, 505 MB, take
// 418 us, 1.2 TB/s.
#include "attn_prompt.h"

namespace beam {

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void beam_attn_prompt_f32(AttnPromptArgs a) {
    using L = Lds<A_F32, D>;
    using S = Stage<A_F32, D>;
    constexpr int TILE = L::TILE;                    // 32 tokens of a step
    constexpr int NQ = D / 8, ND = D / 32;           // 16-byte query pieces per lane, 32-element blocks
    __shared__ __attribute__((aligned(16))) uint8_t sK0[L::BYTES], sV0[L::BYTES], sK1[L::BYTES], sV1[L::BYTES];
    __shared__ int sBad;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int head = blockIdx.x % a.Hkv;
    Block k;
    int part;
    size_t slot;
    if (!block_part(a, k, &part, &slot)) return;
    const int v0 = k.base + part * k.part;
    const int v1 = part + 1 < k.np ? v0 + k.part : k.end;
    const Rows row = rows_of(a, k, wave);
    float4 qf[NQ];
    {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                          (size_t)(k.first + row.qi) * a.qs + (head * a.G + row.qg) * D);
#pragma unroll
        for (int c = 0; c < NQ; ++c) qf[c] = q[2 * c + h];
    }
    const float zs = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;   // reference of the probabilities, this lane's share of their sum
    f32x16 o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = zeros16();

    // The pages of a step's two 16-token blocks, through the scalar cache, two
    // steps ahead.  Blocks past the end look up the last one.
    typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
    const scalar_ints table = (scalar_ints)(uintptr_t)(a.table + (size_t)k.b * a.max_pages);
    const auto token = [&](int place) { return place < k.skip ? place : place + k.gap; };   // of a 16-token block
    const int last16 = (v1 - 1) & ~15;
    const auto page_of = [&](int place) { return table[token(min(place, last16)) >> a.c.pshift]; };
    const auto in_cache = [&](int pg) { return (uint32_t)pg < (uint32_t)a.c.n_pages; };

    S ck, cv;
    const auto load = [&](int v, int pg0, int pg1, uint8_t* sK, uint8_t* sV) {
        const int at = wave * S::ROWS, place = v + (at & ~15), page = at < 16 ? pg0 : pg1;
        const uint8_t *kp, *vp;
        kp = vp = reinterpret_cast<const uint8_t*>(kZeros);
        if (place < v1 && in_cache(page)) {
            const size_t from = (((size_t)page * a.Hkv + head) << a.c.pshift) +
                                ((token(place) + (at & 15)) & ((1 << a.c.pshift) - 1));
            kp = static_cast<const uint8_t*>(a.c.k) + from * S::CB;
            vp = static_cast<const uint8_t*>(a.c.v) + from * S::CB;
        }
        ck.template load<false>(kp, nullptr, sK, at);
        cv.template load<true>(vp, nullptr, sV, at);
    };

    if (threadIdx.x == 0) sBad = -1;
    int pg0 = 0, pg1 = 0, next0 = 0, next1 = 0;
    if (v0 < v1) {
        pg0 = page_of(v0);
        pg1 = page_of(v0 + 16);
        load(v0, pg0, pg1, sK0, sV0);
        next0 = page_of(v0 + TILE);
        next1 = page_of(v0 + TILE + 16);
    }
    // one step: one buffer is worked on while the other fills
    const auto step = [&](int v, uint8_t* sK, uint8_t* sV, uint8_t* oK, uint8_t* oV) {
        __builtin_amdgcn_s_waitcnt(0);   // this wave's loads to LDS have landed
        __syncthreads();                 // everyone's, and no one reads the other buffer any more
        // whether every row of the block, and of the wave, sees all of the step's tokens
        const int ta = token(v), tb = token(v + 16), lo = min(ta, tb), hi = max(ta, tb) + 15;
        const bool have0 = in_cache(pg0), have1 = v + 16 < v1 && in_cache(pg1);
        const auto full = [&](int p0, int p1) {
            return have0 && have1 && v + TILE <= v1 && hi <= p0 && (a.window == 0 || lo > p1 - a.window || hi < a.sinks);
        };
        const bool all = full(k.p0, k.p1), mine = full(row.lo, row.hi);
        if (v + TILE < v1) {
            load(v + TILE, next0, next1, oK, oV);
            pg0 = next0;
            pg1 = next1;
            next0 = page_of(v + 2 * TILE);
            next1 = page_of(v + 2 * TILE + 16);
        }
        const auto sees = [&](int x) {   // whether this lane's row sees token x of the step
            const int tok = (x < 16 ? ta : tb) + (x & 15);
            return (x < 16 ? have0 : have1) && tok <= row.pos &&
                   (a.window == 0 || tok > row.pos - a.window || tok < a.sinks);
        };
        if (!all) mend_values<A_F32, D>(sV, wave, v, &sBad, o, sees);

        // scores: lane (r, h) gets row r, tokens 8 (i / 4) + 4 h + i % 4
        f32x16 z = zeros16();
#pragma unroll
        for (int c = 0; c < NQ; ++c) {
            const float4 kf = *reinterpret_cast<const float4*>(sK + r * L::RB + L::kslot(r, 2 * c + h) * 16);
            z = __builtin_amdgcn_mfma_f32_32x32x2f32(kf.x, qf[c].x, z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_32x32x2f32(kf.y, qf[c].y, z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_32x32x2f32(kf.z, qf[c].z, z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_32x32x2f32(kf.w, qf[c].w, z, 0, 0, 0);
        }
        if (!mine) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = sees(8 * (i / 4) + 4 * h + i % 4) ? z[i] : -INFINITY;
        }
        // The reference moves (and what was summed is rescaled) only when a
        // score exceeds it by 8 powers of two.
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, z[i]);
        top *= zs;
        if (__any(top > m + 8.f)) {
            const float mn = fmaxf(m, max_halves(top));
            // before the first score the sums are 0, or infinite by mend_values
            const float alpha = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[t][i] *= alpha;
        }
        const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = __builtin_amdgcn_exp2f(fmaf(z[i], zs, -ms));
#pragma unroll
        for (int i = 0; i < 16; i += 4) l += (z[i] + z[i + 1]) + (z[i + 2] + z[i + 3]);
        // values: a lane's element 32 t + r of the token that its probability is of
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int vr = 8 * (i / 4) + 4 * h + i % 4, e = 32 * t + r;
                const float x = *reinterpret_cast<const float*>(sV + vr * L::RB + L::vslot(vr, e / 4) * 16 + e % 4 * 4);
                o[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, z[i], o[t], 0, 0, 0);
            }
    };
    for (int v = v0; v < v1; v += 2 * TILE) {
        step(v, sK0, sV0, sK1, sV1);
        if (v + TILE < v1) step(v + TILE, sK1, sV1, sK0, sV0);
    }
    write_rows<A_F32, D>(a, k, row, slot, head, wave, o, m, l, l);
}

hipError_t launch_attn_prompt_f32(const AttnPromptArgs& a, hipStream_t st) {
    if (a.D == 64) return launch_prompt<A_F32, 64>(beam_attn_prompt_f32<64>, a, st);
    if (a.D == 128) return launch_prompt<A_F32, 128>(beam_attn_prompt_f32<128>, a, st);
    return launch_prompt<A_F32, 256>(beam_attn_prompt_f32<256>, a, st);
}

}  // namespace beam
