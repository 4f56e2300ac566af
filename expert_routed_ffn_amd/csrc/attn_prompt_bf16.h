// The attention of new tokens over caches that are bf16 in LDS: bf16, e4m3 and 4
// bits.
#pragma once

#include "attn_prompt.h"

namespace beam {

// A wave works on 32 tokens at a time, in three stages a step apart: the scores
// of block u (first product), the probabilities of block u - 1, the weighted sum
// of the values of block u - 2 (second product).  A step's 2 D / 16 matrix
// instructions and its softmax do not depend on each other, so that they are
// interleaved one for one and the matrix cores have work while the vector unit
// has.  A tile of 64 tokens is two blocks: the workgroup meets once per tile t,
// when the keys of tile t and the values of tile t - 1 have landed in LDS, and
// then starts the loads of the keys of tile t + 1 and the values of tile t.
// (One stage after the other, 16384 tokens: 3.47 ms, so 3.28 then; e4m3, 4096 tokens:
// 368 and 253 us.  Two workgroups per CU hold 64 KB of LDS each at D = 128, of two
// waves per SIMD; at D = 256 a workgroup has 128 KB and the CU to itself.  Blocks
// of 256 rows on eight waves are 1 to 7 % faster at 16384 tokens and slower below.)
// A probability enters the second product as one rounded bf16, off by 2^-8 of
// itself at most; over many tokens this cancels in part (results are 2.0 to 2.3e-3
// from the formula's in the mean square, 1.66e-3 of it their own rounding), and
// where values are equal in whole, since the sum is of the rounded ones.  With
// e4m3, where the value rows' scales enter first, it is of them as they are.  Two
// operands, as in decode, are half as many matrix instructions again.
template <int KIND, int D, bool FEW>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void beam_attn_prompt(AttnPromptArgs a) {
    using L = Lds<KIND, D>;
    using S = Stage<KIND, D>;
    constexpr int TILE = L::TILE;                    // 64 tokens
    constexpr int NM = D / 16, ND = D / 32;          // matrix instructions of a product per block
    constexpr bool SC = KIND == A_FP8;               // scale per row
    // two buffers each, variables of their own: so the compiler sees that reads
    // of one need not wait for loads into the other
    __shared__ __attribute__((aligned(16))) uint8_t sK0[L::BYTES], sV0[L::BYTES], sK1[L::BYTES], sV1[L::BYTES];
    // of tile t at t % 4: e4m3 scales, and which waves' rows there are (a byte each)
    __shared__ __attribute__((aligned(16))) float sKs[4][SC ? TILE : 4], sVs[4][SC ? TILE : 4];
    __shared__ uint32_t sThere[4];
    __shared__ float sJoin[2][3][FEW ? 64 : 1];
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
    const int tiles = (v1 - v0 + TILE - 1) / TILE;
    // FEW: of a block of up to 64 rows waves 0, 1 take the rows with the first 32
    // tokens of a tile, waves 2, 3 with the others, and are joined at the end.  Half
    // the waves would be idle else: bf16, 4 sequences of 8 drafted tokens over
    // 32768 in the last-level cache, 67.7 -> 56.6 us; 200 single tokens and 4 chunks
    // over e4m3 152 -> 119.
    // Both loops in one kernel cost long prompts registers (16384 tokens 3.30 ->
    // 3.37 ms, e4m3 windows 170 -> 197 us), so those have one without.  At D = 256
    // it gains nothing (35.6 -> 36.0 us at 16 of 64 tokens).
    const bool halves = FEW && k.row1 - k.row0 <= 64;
    const int rg = halves ? wave & 1 : wave, ts = halves ? wave >> 1 : 0;
    const Rows row = rows_of(a, k, rg);
    bf16x8 qf[NM];
    {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                        (size_t)(k.first + row.qi) * a.qs + (head * a.G + row.qg) * D);
#pragma unroll
        for (int c = 0; c < NM; ++c) qf[c] = __builtin_bit_cast(bf16x8, q[2 * c + h]);
    }
    const float zs = a.scale * kLog2e;
    // Reference that the probabilities are relative to, and this lane's share of
    // their sum: as they enter the second product, rounded, so that the rounding
    // cancels and equal values come back as themselves (e4m3: as they are), and as
    // they are, for lse.
    constexpr bool BF = !SC;
    float m = -INFINITY, l = 0.f, lx = 0.f;
    f32x16 o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = zeros16();

    // A wave stages one 16-token block of a tile; its page is looked up through
    // the scalar cache two tiles ahead.  Blocks past the end look up the last one.
    typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
    const scalar_ints table = (scalar_ints)(uintptr_t)(a.table + (size_t)k.b * a.max_pages);
    const auto token = [&](int place) { return place < k.skip ? place : place + k.gap; };   // of a 16-token block
    const int last16 = (v1 - 1) & ~15;
    const auto page_of = [&](int t) { return table[token(min(v0 + t * TILE + wave * 16, last16)) >> a.c.pshift]; };
    // the wave's rows of a tile in the cache; negative: there are none
    const auto rows_at = [&](int t, int page) -> int64_t {
        const int place = v0 + t * TILE + wave * 16;
        if (place >= v1 || (uint32_t)page >= (uint32_t)a.c.n_pages) return -1;
        return (((int64_t)page * a.Hkv + head) << a.c.pshift) + (token(place) & ((1 << a.c.pshift) - 1));
    };
    constexpr int SB = KIND == A_FP4 ? D / 32 : 4;   // scale bytes per row
    const auto side = [&](const void* p, int64_t at, int bytes) {
        const uint64_t x = (uint64_t)(at < 0 ? reinterpret_cast<const uint8_t*>(kZeros)
                                             : static_cast<const uint8_t*>(p) + at * bytes);
        return reinterpret_cast<const uint8_t*>(   // in scalar registers
            (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
            (uint32_t)__builtin_amdgcn_readfirstlane((int)x));
    };
    S ck, cv;
    float ksc = 0.f, vsc = 0.f;
    const auto load_keys = [&](int t, int64_t at, uint8_t* sK) {
        const uint8_t* scales = side(a.c.ks, at, SB);
        ck.template load<false>(side(a.c.k, at, S::CB), scales, sK, wave * 16);
        if constexpr (SC) {   // the values' too: they enter the probabilities
            ksc = reinterpret_cast<const float*>(scales)[lane & 15];
            vsc = reinterpret_cast<const float*>(side(a.c.vs, at, SB))[lane & 15];
        }
        if (lane == 0) reinterpret_cast<uint8_t*>(&sThere[t & 3])[wave] = at >= 0;
    };
    const auto store_keys = [&](int t, uint8_t* sK) {
        ck.template store<false>(sK, wave * 16);
        if constexpr (SC) {
            if (lane < 16) {
                sKs[t & 3][wave * 16 + lane] = ksc;
                sVs[t & 3][wave * 16 + lane] = vsc;
            }
        }
    };
    const auto load_values = [&](int64_t at, uint8_t* sV) {
        cv.template load<true>(side(a.c.v, at, S::CB), side(a.c.vs, at, SB), sV, wave * 16);
    };

    // Byte places in LDS of this lane's key piece 2 c + h of row r, and of its four
    // value elements for a transposing read: the exchange of pieces is an
    // exclusive or, so piece and block enter by one.
    const int i16 = lane & 15;
    int kat = r * L::RB + L::kslot(r, h) * 16;       // ^ 32 c
    int vat = (4 * h + i16 / 4) * L::RB +
              L::vslot(4 * h + i16 / 4, (lane & 16) / 8 + i16 % 4 / 2) * 16 + i16 % 2 * 8;   // ^ (64 t + 32 y), + (16 s + 8 y) RB

    // What a row sees of a tile: its 16-token blocks' first tokens, which are there.
    struct Tile {
        int v;
        uint32_t there;
        bool all, mine;      // every row of the block, of the wave, sees all of it
    };
    const auto tile_of = [&](int t) {
        Tile x;
        x.v = v0 + t * TILE;
        x.there = __builtin_amdgcn_readfirstlane(sThere[t & 3]);
        const int lo = token(x.v), hi = lo + TILE - 1;
        const bool ok = x.there == 0x01010101u && x.v + TILE <= v1 && (x.v >= k.skip || x.v + TILE <= k.skip);
        x.all = ok && hi <= k.p0 && (a.window == 0 || lo > k.p1 - a.window || hi < a.sinks);
        x.mine = ok && hi <= row.lo && (a.window == 0 || lo > row.hi - a.window || hi < a.sinks);
        return x;
    };
    // which of the 16 tokens of block u of a tile this lane's row sees, as bits
    const auto seen16 = [&](const Tile& x, int u) {
        const int t0 = token(x.v + 16 * u);
        const auto below = [](int n) { return (1 << min(max(n, 0), 16)) - 1; };   // bits 0 .. n - 1
        int bits = below(row.pos - t0 + 1);
        if (a.window > 0) bits &= ~below(row.pos - a.window + 1 - t0) | below(a.sinks - t0);
        return x.there >> (8 * u) & 1 ? bits : 0;
    };

    // One step.  QK: scores zo from the keys at kp.  SM: probabilities po from the
    // scores zi of half `half` of tile x.  PV: sums of the values at vp with pi.
    const auto step = [&](auto QK, auto SM, auto PV, const uint8_t* kp, const uint8_t* vp, f32x16& zo, f32x16& zi,
                          const uint32_t (&pi)[8], uint32_t (&po)[8], const Tile& x, int t,
                          int half) __attribute__((always_inline)) {
        // Pieces of keys and values are read two matrix instructions ahead, the
        // first ones before the softmax's reference is looked at.
        uint4 kf[2], vf[2];
        const auto key = [&](int j) { return *reinterpret_cast<const uint4*>(kp + (kat ^ (32 * j))); };
        const auto value = [&](int j) {
            // elements 32 e + lane % 32, tokens 16 s + 8 y + 4 h + 0 .. 3: the 16 lanes
            // of a group read four rows of 16 elements, lane i row i / 4 and elements
            // 4 (i % 4) .. + 3, and get element i of each
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            const int e = j / 2, s = j % 2;
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint8_t* p = vp + (vat ^ (64 * e + 32 * y)) + (16 * s + 8 * y) * L::RB;
                const uint2 u = __builtin_bit_cast(
                    uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
                w[2 * y] = u.x;
                w[2 * y + 1] = u.y;
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        if constexpr (D == 256) asm volatile("" : "+v"(kat), "+v"(vat));   // places are formed anew: no registers to hold them
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (QK()) kf[j] = key(j);
            if constexpr (PV()) vf[j] = value(j);
        }
        float alpha = 1.f, ms = 0.f;
        int moved = 0;
        float4 vs[4];
        if constexpr (SM()) {
            if constexpr (SC) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int y = 32 * half + 2 * i + 4 * h;
                    const float4 f = *reinterpret_cast<const float4*>(&sKs[t & 3][y]);
                    zi[i] *= f.x; zi[i + 1] *= f.y; zi[i + 2] *= f.z; zi[i + 3] *= f.w;
                    vs[i / 4] = *reinterpret_cast<const float4*>(&sVs[t & 3][y]);
                }
            }
            if (__builtin_expect(!x.mine, 0)) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {        // its 16-token blocks
                    const int live = seen16(x, 2 * half + u) >> (4 * h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // all ones where bit 8 (i / 4) + i % 4 is set, else zeros: -inf there
                        const int on = __builtin_amdgcn_sbfe(live, 8 * (i / 4) + i % 4, 1);
                        const int z = (int)__float_as_uint(zi[8 * u + i]);
                        zi[8 * u + i] = __uint_as_float((uint32_t)((z & on) | (0xFF800000 & ~on)));
                        if constexpr (SC) {   // its scale may be NaN
                            float* f = reinterpret_cast<float*>(&vs[2 * u + i / 4]) + i % 4;
                            *f = __uint_as_float(__float_as_uint(*f) & (uint32_t)on);
                        }
                    }
                }
            }
            // The reference moves (and what was summed is rescaled) only when a
            // score exceeds it by 8 powers of two.
            float top = fmaxf(zi[0], zi[1]);
#pragma unroll
            for (int i = 2; i < 16; i += 2) top = fmaxf(fmaxf(top, zi[i]), zi[i + 1]);
            top *= zs;
            moved = __any(top > m + 8.f);
            if (__builtin_expect(moved, 0)) {
                const float mn = fmaxf(m, max_halves(top));
                // before the first score the sums are 0, or infinite by mend_values
                alpha = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= alpha;
                lx *= alpha;
            }
            ms = m == -INFINITY ? 0.f : m;
            // not known to be the same below: the instructions between stay one stretch
            moved = __builtin_amdgcn_readfirstlane(moved);
            asm volatile("" : "+s"(moved));
        }
        if constexpr (QK()) zo = zeros16();
#pragma unroll
        for (int j = 0; j < NM; ++j) {
            if constexpr (QK()) {
                zo = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[j % 2]), qf[j], zo, 0, 0, 0);
                if (j + 2 < NM) kf[j % 2] = key(j + 2);
            }
            if constexpr (PV()) {
                const int s = j % 2;
                o[j / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, vf[j % 2]),
                    __builtin_bit_cast(bf16x8, make_uint4(pi[4 * s], pi[4 * s + 1], pi[4 * s + 2], pi[4 * s + 3])),
                    o[j / 2], 0, 0, 0);
                if (j + 2 < NM) vf[j % 2] = value(j + 2);
            }
            if constexpr (SM()) {
                constexpr int E = 16 / NM;           // scores of this piece
#pragma unroll
                for (int i = j * E; i < j * E + E; ++i) zi[i] = __builtin_amdgcn_exp2f(fmaf(zi[i], zs, -ms));
#pragma unroll
                for (int i = (j * E) & ~1; i + 1 < j * E + E; i += 2) {
                    float y0 = zi[i], y1 = zi[i + 1];
                    (SC ? l : lx) += y0 + y1;
                    if constexpr (SC) {
                        const float* f = reinterpret_cast<const float*>(&vs[i / 4]) + i % 4;
                        y0 *= f[0];
                        y1 *= f[1];
                    }
                    po[i / 2] = pack_bf16x2(y0, y1);
                    if constexpr (BF) {
                        typedef __bf16 pair __attribute__((ext_vector_type(2)));
                        const pair one = {(__bf16)1.f, (__bf16)1.f};
                        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair, po[i / 2]), one, l, false);
                    }
                }
            }
        }
        if constexpr (SM()) {
#pragma unroll
            for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(po[i]));   // the probabilities are formed here, not where they are used
            asm volatile("" : "+v"(l), "+v"(lx));
            if (__builtin_expect(moved, 0)) {
#pragma unroll
                for (int e = 0; e < ND; ++e)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[e][i] *= alpha;
            }
        }
    };

    const std::true_type yes;
    const std::false_type no;
    f32x16 zA = zeros16(), zB;
    uint32_t pA[8], pB[8];
    Tile before{}, now{};
    int64_t at = -1, at_next = -1;                   // the wave's rows of tiles t and t + 1
    int page = 0;                                    // of tile t + 2
    if (threadIdx.x == 0) sBad = -1;
    if (tiles > 0) {
        at_next = rows_at(0, page_of(0));
        load_keys(0, at_next, sK0);
        page = page_of(1);
        store_keys(0, sK0);
    }
    // tile t: keys at sK, the values of tile t - 1 at sV; oK and oV fill
    const auto turn = [&](int t, auto HALVES, auto FIRST, auto LAST, uint8_t* sK, uint8_t* sV, uint8_t* oK,
                          uint8_t* oV) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0);   // this wave's loads to LDS have landed
        __syncthreads();                 // everyone's, and no one reads the other buffers any more
        if constexpr (!LAST()) {
            now = tile_of(t);
            at = at_next;
            load_values(at, oV);
            if (t + 1 < tiles) {
                at_next = rows_at(t + 1, page);
                load_keys(t + 1, at_next, oK);
                page = page_of(t + 2);
            }
        }
        if constexpr (!FIRST())
            if (__builtin_expect(!before.all, 0))
                mend_values<KIND, D>(sV, wave, t, &sBad, o, [&](int y) {
                    if (HALVES() && y / 32 != ts) return false;
                    return (seen16(before, y / 16) >> (y & 15) & 1) != 0;
                });
        if constexpr (HALVES()) {
            const uint8_t *kh = sK + ts * 32 * L::RB, *vh = sV + ts * 32 * L::RB;
            if constexpr (LAST()) {
                step(no, no, yes, kh, vh, zB, zA, pA, pB, before, t - 1, 0);
            } else {
                if constexpr (FIRST()) step(yes, no, no, kh, vh, zB, zA, pA, pB, before, t - 1, 0);
                else step(yes, no, yes, kh, vh, zB, zA, pA, pB, before, t - 1, 0);
                step(no, yes, no, kh, vh, zA, zB, pB, pA, now, t, ts);
            }
        } else if constexpr (FIRST()) {
            step(yes, no, no, sK, sV, zB, zA, pA, pB, before, t - 1, 1);
            step(yes, yes, no, sK + 32 * L::RB, sV, zA, zB, pB, pA, now, t, 0);
        } else if constexpr (LAST()) {
            step(no, yes, yes, sK, sV, zB, zA, pA, pB, before, t - 1, 1);
            step(no, no, yes, sK, sV + 32 * L::RB, zA, zB, pB, pA, now, t, 0);
        } else {
            step(yes, yes, yes, sK, sV, zB, zA, pA, pB, before, t - 1, 1);
            step(yes, yes, yes, sK + 32 * L::RB, sV + 32 * L::RB, zA, zB, pB, pA, now, t, 0);
        }
        if constexpr (!LAST()) {
            cv.template store<true>(oV, wave * 16);
            if (t + 1 < tiles) store_keys(t + 1, oK);
            before = now;
        }
    };
    // tile t's keys are in buffer t % 2, its values too: they are loaded in turn t
    // and used in turn t + 1
    if (FEW && halves && tiles > 0) {
        if constexpr (FEW) {
            turn(0, yes, yes, no, sK0, sV1, sK1, sV0);
            int t = 1;
            for (; t + 1 < tiles; t += 2) {
                turn(t, yes, no, no, sK1, sV0, sK0, sV1);
                turn(t + 1, yes, no, no, sK0, sV1, sK1, sV0);
            }
            if (t < tiles) {
                turn(t, yes, no, no, sK1, sV0, sK0, sV1);
                turn(t + 1, yes, no, yes, sK0, sV1, sK1, sV0);
            } else {
                turn(t, yes, no, yes, sK1, sV0, sK0, sV1);
            }
        }
    } else if (tiles > 0) {
        turn(0, no, yes, no, sK0, sV1, sK1, sV0);
        int t = 1;
        for (; t + 1 < tiles; t += 2) {
            turn(t, no, no, no, sK1, sV0, sK0, sV1);
            turn(t + 1, no, no, no, sK0, sV1, sK1, sV0);
        }
        if (t < tiles) {
            turn(t, no, no, no, sK1, sV0, sK0, sV1);
            turn(t + 1, no, no, yes, sK0, sV1, sK1, sV0);
        } else {
            turn(t, no, no, yes, sK1, sV0, sK0, sV1);
        }
    }
    if (halves) {
        // waves 2 and 3 hand over what they have, lane by lane, in the tiles' memory
        static_assert(L::BYTES == 32 * D * sizeof(float), "a wave's sums fit a tile");
        float* mem = reinterpret_cast<float*>(rg ? sV0 : sK0) + lane;
        __syncthreads();
        if (ts) {
#pragma unroll
            for (int e = 0; e < ND; ++e)
#pragma unroll
                for (int i = 0; i < 16; ++i) mem[(16 * e + i) * 64] = o[e][i];
            sJoin[rg][0][lane] = m;
            sJoin[rg][1][lane] = l;
            sJoin[rg][2][lane] = lx;
        }
        __syncthreads();
        if (ts) return;
        const float m1 = sJoin[rg][0][lane], mn = fmaxf(m, m1), ms = mn == -INFINITY ? 0.f : mn;
        const float f0 = __builtin_amdgcn_exp2f(m - ms), f1 = __builtin_amdgcn_exp2f(m1 - ms);
        m = mn;
        l = fmaf(f1, sJoin[rg][1][lane], f0 * l);
        lx = fmaf(f1, sJoin[rg][2][lane], f0 * lx);
#pragma unroll
        for (int e = 0; e < ND; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[e][i] = fmaf(f1, mem[(16 * e + i) * 64], f0 * o[e][i]);
    }
    write_rows<KIND, D>(a, k, row, slot, head, rg, o, m, l, BF ? lx : l);
}

template <int KIND> hipError_t launch_prompt_d(const AttnPromptArgs& a, hipStream_t st) {
    if (a.D == 64)
        return launch_prompt<KIND, 64>(a.p.few ? beam_attn_prompt<KIND, 64, true> : beam_attn_prompt<KIND, 64, false>,
                                       a, st);
    if (a.D == 128)
        return launch_prompt<KIND, 128>(
            a.p.few ? beam_attn_prompt<KIND, 128, true> : beam_attn_prompt<KIND, 128, false>, a, st);
    return launch_prompt<KIND, 256>(beam_attn_prompt<KIND, 256, false>, a, st);
}

}  // namespace beam
