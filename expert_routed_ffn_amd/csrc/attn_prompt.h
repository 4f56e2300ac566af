// Attention of any number of new tokens per sequence over a paged key-value
// cache: causal, sliding window, first tokens that stay visible (sinks).
//
// The new tokens of a sequence and the G query heads of a key-value head form
// n * G rows, token by token, cut into blocks of 128 for a workgroup of four
// waves: a block's rows are few tokens, so that its causal and window edges are
// narrow whatever n is.  A wave holds 32 rows as the columns of
//   Z^T [tokens, 32] = K Q^T     and     O^T [D, 32] = V^T P^T
// with one pass over the tokens and the running maximum and sum of the softmax
// beside them.  Of a product's 32 x 32 result lane (r, h) holds column r and
// rows 8 (i / 4) + 4 h + i % 4, i = 0 .. 15: so a query's scores lie in two
// lanes, its maximum, sum and rescaling are a lane's own, and eight scores in a
// row of i are the second product's right operand where its reduction index
// (h, j) stands for token 8 (j / 4) + 4 h + j % 4 of 16.  The probabilities move
// between no lanes; V^T comes out of LDS by the transposing reads.
//
// Keys and values of a step (64 tokens) go to LDS as bf16, once for the four
// waves: by direct loads from a bf16 cache, through registers from an 8- or 4-bit
// one, the next step's while this one is worked on.
//
// 4 D flops per row and visible token over keys and values that 128 rows share:
// the matrix cores bound it where prompts are long, with the vector unit beside
// them (softmax, LDS and staging), HBM where few rows meet a long cache, latency
// where there is little of both.  48 heads over 8 of 128, bf16: 16384 tokens 3.28 to
// 3.38 ms, 976 to 1005 TFLOP/s (a large product reaches 1343); 2048 tokens 66 to 77
// us, where workgroups of 1 to 32 tiles do not fill the chip evenly; 4 x 8 tokens
// over up to 32768 72 us, 3.5 TB/s (253 MB, from HBM; 56 us from the last-level cache, which
// holds them), on 416 of the 512 workgroups that the chip holds; 37 tokens 7 us.
// e4m3, 4096 tokens: 252 us, 4 bits 240, bf16 228.
#pragma once

#include "attn_common.h"

namespace beam {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPromptWaves = kPromptRows / 32;
constexpr int kPromptMinPart = 256;     // tokens of a part, at least
constexpr int kPromptRound = 64;

// ---------------------------------------------------------------- what a block sees

// Rows [row0, row1) of the n * G rows of sequence b, whose queries stand at
// positions p0 .. p1; they see places [base, end) of the sequence: its tokens
// without the 16-token blocks that neither sinks nor window reach, token =
// place + (place < skip ? 0 : gap).
struct Block {
    int b, first, n, len;    // sequence, its first new token's row of q, new tokens, length
    int row0, row1, p0, p1;
    int base, end, skip, gap;
    int part, np;            // places per part, parts
};

BEAM_DEV int prompt_offset(const AttnPromptArgs& a, int b) { return min(max(a.offsets[b], 0), a.T); }

// places that the rows of positions p0 .. p1 see
BEAM_DEV void block_span(const AttnPromptArgs& a, Block& k) {
    const int start = a.window > 0 ? max(0, k.p0 - a.window + 1) : 0;
    k.base = start & ~15;
    const int sinks = min(a.sinks, start);
    k.skip = (sinks + 15) & ~15;
    k.gap = 0;
    if (sinks > 0) {
        k.gap = max(0, k.base - k.skip);
        k.base = 0;
    }
    k.end = max(k.p1 + 1 - k.gap, k.base);
}

// Sequence b with its block number `at` (false: it has no such block).  Blocks
// of all sequences are numbered with gaps: those of sequence b from
// floor(first row / 128) + b on, which leaves room for its last, short one.
BEAM_DEV bool block_of(const AttnPromptArgs& a, int b, int at, Block& k) {
    k.b = b;
    k.first = prompt_offset(a, b);
    k.n = prompt_offset(a, b + 1) - k.first;
    k.row0 = at * kPromptRows;
    if (k.n <= 0 || at < 0 || k.row0 >= k.n * a.G) return false;
    k.row1 = min(k.row0 + kPromptRows, k.n * a.G);
    const int cap = (int)min((int64_t)a.max_pages << a.c.pshift, (int64_t)kMaxLen);
    k.len = min(max(a.lens[b], 0), cap);
    k.p0 = k.len - k.n + k.row0 / a.G;
    k.p1 = k.len - k.n + (k.row1 - 1) / a.G;
    block_span(a, k);
    // parts: the sequence's last block sees the most places; even parts of them
    k.part = 1 << 30;
    if (a.p.S > 1 && (a.p.every || k.n * a.G <= kPromptRows)) {
        Block last = k;
        last.p0 = k.len - k.n + (k.n * a.G - 1) / kPromptRows * kPromptRows / a.G;
        last.p1 = k.len - 1;
        block_span(a, last);
        const uint32_t all = (uint32_t)(last.end - last.base) + 16;
        k.part = (int)max((all + a.p.S - 1) / a.p.S, (uint32_t)kPromptMinPart);
        k.part = (k.part + kPromptRound - 1) & ~(kPromptRound - 1);
    }
    k.np = max((int)((uint32_t)(k.end - k.base + k.part - 1) / (uint32_t)k.part), 1);
    k.np = min(k.np, (int)a.p.S);               // the last part takes the rest
    return true;
}

// First block number of sequence b.
BEAM_DEV int first_block(const AttnPromptArgs& a, int b) {
    return (int)((int64_t)prompt_offset(a, b) * a.G / kPromptRows) + b;
}

// The sequence of block number idx: 64 candidates at a time, one per lane.
BEAM_DEV int sequence_of(const AttnPromptArgs& a, int idx) {
    int lo = 0, n = a.B;   // first_block(lo) <= idx; candidates lo .. lo + n - 1
    const int lane = threadIdx.x & 63;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int cand = lo + lane * step;
        const bool before = cand < lo + n && first_block(a, cand) <= idx;
        const int k = max(__popcll(__ballot(before)) - 1, 0);   // ascending: the first k + 1 lanes
        const int next = lo + k * step;
        n = min(step, lo + n - next);
        lo = next;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// ---------------------------------------------------------------- LDS

// Rows of D elements in 16-byte pieces, a piece's place exchanged by its row so
// that the lanes of one access spread over the banks: keys are read 16 rows at a
// time in one column of pieces, values four rows at a time in four.
template <int KIND, int D> struct Lds {
    static constexpr int ES = KIND == A_F32 ? 4 : 2;
    static constexpr int TILE = KIND == A_F32 ? 32 : 64;
    static constexpr int RB = D * ES, NP = RB / 16;
    static constexpr int BYTES = TILE * RB;
    static BEAM_DEV int kslot(int row, int piece) {
        if constexpr (NP == 8) return piece ^ ((row >> 1) & 7);
        return piece ^ (row & 15);
    }
    static BEAM_DEV int vslot(int row, int piece) {
        if constexpr (KIND == A_F32) return piece ^ (((row >> 2) & 1) << 3);
        if constexpr (NP == 8) return piece ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3));
        return piece ^ (((row & 3) << 2) | ((row >> 2) & 3));
    }
};

// As many zeros as the rows that a wave stages: what a 16-token block past the
// end or on a bad page is read from.
__device__ const uint4 kZeros[512] = {};

BEAM_DEV void to_lds(const void* src, void* dst) {   // dst: the wave's, lane i's 16 bytes at 16 i
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)src,
                                     (__attribute__((address_space(3))) uint32_t*)dst, 16, 0, 0);
}

// A step's keys or values on their way to LDS: what a wave's lanes load of its
// TILE / 4 rows, all in one 16-token block.
template <int KIND, int D> struct Stage {
    using L = Lds<KIND, D>;
    static constexpr int ROWS = L::TILE / kPromptWaves;   // 16, fp32: 8
    static constexpr bool DIRECT = KIND == A_F32 || KIND == A_BF16;
    static constexpr int CB = KIND == A_F32 ? 4 * D : (KIND == A_BF16 ? 2 * D : (KIND == A_FP8 ? D : D / 2));   // cache row
    static constexpr int N = (ROWS * CB / 16 + 63) / 64;   // 16-byte loads per lane
    uint4 w[DIRECT ? 1 : N];
    uint32_t s[KIND == A_FP4 ? N : 1];   // FP4: scale bytes

    // rows at `src` (the same for the wave) to rows row0 .. of the LDS tile
    template <bool IS_V> BEAM_DEV void load(const uint8_t* src, const uint8_t* scales, uint8_t* tile, int row0) {
        int lane = threadIdx.x & 63;
        // D = 256: places are formed anew for each tile, not held in registers: those
        // that spilled waited for the loads in flight (4096 tokens, 32 heads over 4,
        // bf16 489 -> 371 us, 4 bits 491 -> 444, e4m3 562 -> 547; at D = 128, where
        // nothing spills in the loop, it costs 3 to 5 %)
        if constexpr (D == 256) asm volatile("" : "+v"(lane));
        if constexpr (DIRECT) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = i * 64 + lane, row = row0 + p / L::NP;
                const int piece = IS_V ? L::vslot(row, p % L::NP) : L::kslot(row, p % L::NP);
                to_lds(src + (uint32_t)((p / L::NP) * CB + piece * 16), tile + row0 * L::RB + i * 1024);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t p = min(i * 64 + lane, ROWS * CB / 16 - 1);
                w[i] = *reinterpret_cast<const uint4*>(src + p * 16);
                if constexpr (KIND == A_FP4) s[i] = scales[p];   // 16 bytes are a block of 32
            }
        }
    }
    // and from registers into the tile, as bf16 (exact)
    template <bool IS_V> BEAM_DEV void store(uint8_t* tile, int row0) {
        if constexpr (!DIRECT) {
            constexpr int PR = CB / 16;                    // loads per row
            constexpr int EP = KIND == A_FP8 ? 2 : 4;      // LDS pieces per load
            int lane = threadIdx.x & 63;
            if constexpr (D == 256) asm volatile("" : "+v"(lane));   // places are formed anew, not held
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = i * 64 + lane;
                if (p >= ROWS * PR) continue;
                const int row = row0 + p / PR, piece = p % PR * EP;
                const uint32_t c[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < EP; ++e) {
                    uint4 v;
                    if constexpr (KIND == A_FP8) {
                        v = make_uint4(e4m3_lo(c[2 * e]), e4m3_hi(c[2 * e]), e4m3_lo(c[2 * e + 1]), e4m3_hi(c[2 * e + 1]));
                    } else {
                        const float f = e8m0(s[i]);
                        v = make_uint4(e2m1_pair<0>(c[e], f), e2m1_pair<1>(c[e], f), e2m1_pair<2>(c[e], f),
                                       e2m1_pair<3>(c[e], f));
                    }
                    const int slot = IS_V ? L::vslot(row, piece + e) : L::kslot(row, piece + e);
                    *reinterpret_cast<uint4*>(tile + row * L::RB + slot * 16) = v;
                }
            }
        }
    }
};

// ---------------------------------------------------------------- rows

BEAM_DEV float max_halves(float v) {
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
BEAM_DEV float sum_halves(float v) {
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
BEAM_DEV f32x16 zeros16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// A wave's 32 rows, one to a lane: lanes r and r + 32 hold row r.  Rows past the
// block's last repeat it.
struct Rows {
    int qi, qg, pos;         // query token and head of this lane's row, its position
    int lo, hi;              // the wave's first and last position
    bool live;
};
BEAM_DEV Rows rows_of(const AttnPromptArgs& a, const Block& k, int wave) {
    const int r = threadIdx.x & 31, w0 = k.row0 + wave * 32, end = k.row1 - 1;
    Rows x;
    const int row = min(w0 + r, end);
    x.qi = row / a.G;
    x.qg = row - x.qi * a.G;
    x.pos = k.len - k.n + x.qi;
    x.lo = k.len - k.n + min(w0, end) / a.G;
    x.hi = k.len - k.n + min(w0 + 31, end) / a.G;
    x.live = w0 + r < k.row1;
    return x;
}

// The workgroup's block, its part of it and that part's place in the workspace;
// false: there is none.  Parts 1 .. of the sequences in one block come first, then
// the blocks, a sequence's last ones, which see most, first.
BEAM_DEV bool block_part(const AttnPromptArgs& a, Block& k, int* part, size_t* slot) {
    const int at = blockIdx.x / a.Hkv, S = (int)a.p.S;
    int idx = (int)a.p.blocks - 1 - at, s = 0;
    if (a.p.every) {
        s = blockIdx.y;
    } else {
        const int extra = a.B * (S - 1);
        if (at < extra) {
            s = 1 + at % (S - 1);
            *part = s;
            *slot = (size_t)(at / (S - 1)) * S + s;
            return block_of(a, at / (S - 1), 0, k) && s < k.np;
        }
        idx += extra;
    }
    const int b = sequence_of(a, idx);
    if (!block_of(a, b, idx - first_block(a, b), k)) return false;
    *part = s;
    *slot = (size_t)(a.p.every ? idx : b) * S + s;
    return s < k.np;
}

// The value rows of a wave in LDS, rows row0 .. of a tile: whether an element is
// not finite; SET: 0 in its place.
template <int KIND, int D, bool SET> BEAM_DEV bool find_not_finite(uint8_t* tile, int row0) {
    using L = Lds<KIND, D>;
    bool bad = false;
    for (int i = threadIdx.x & 63; i < L::TILE / kPromptWaves * L::NP; i += 64) {
        uint4* w = reinterpret_cast<uint4*>(tile + row0 * L::RB + i * 16);
        uint32_t x[4] = {w->x, w->y, w->z, w->w};
        bool here = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if ((x[e] & 0x7F800000u) == 0x7F800000u) {
                x[e] &= KIND == A_F32 ? 0u : 0x0000FFFFu;
                here = true;
            }
            if (KIND != A_F32 && (x[e] & 0x7F80u) == 0x7F80u) {
                x[e] &= 0xFFFF0000u;
                here = true;
            }
        }
        if (SET && here) *w = make_uint4(x[0], x[1], x[2], x[3]);
        bad |= here;
    }
    return bad;
}

// A value that is not finite must not reach rows that do not see it: 0 times it
// is NaN.  Where rows differ in what they see of a tile, all waves look its
// values through first (`tag` tells the tiles apart).  If one is not finite, it
// is added to the sums of the rows that see it, with any weight, and is 0 in LDS
// from there on.  sees(x): whether this lane's row sees token x of the tile.
template <int KIND, int D, typename Sees>
BEAM_DEV void mend_values(uint8_t* tile, int wave, int tag, int* flag, f32x16 (&o)[D / 32], Sees sees) {
    using L = Lds<KIND, D>;
    const int lane = threadIdx.x & 63, h = lane >> 5, row0 = wave * (L::TILE / kPromptWaves);
    if (__any(find_not_finite<KIND, D, false>(tile, row0)) && lane == 0) *flag = tag;
    __syncthreads();
    if (*flag != tag) return;
#pragma unroll 1
    for (int y = 0; y < L::TILE; ++y) {
        const bool add = sees(y);
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int e = 32 * t + 2 * i + 4 * h;
                const uint8_t* w = tile + y * L::RB + L::vslot(y, e * L::ES / 16) * 16 + e * L::ES % 16;
                float x[4];
                if constexpr (KIND == A_F32) {
                    const float4 f = *reinterpret_cast<const float4*>(w);
                    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
                } else {
                    const uint2 f = *reinterpret_cast<const uint2*>(w);
                    x[0] = __uint_as_float(f.x << 16); x[1] = __uint_as_float(f.x & 0xFFFF0000u);
                    x[2] = __uint_as_float(f.y << 16); x[3] = __uint_as_float(f.y & 0xFFFF0000u);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)   // x - x: 0, or NaN
                    o[t][i + j] += (add & (x[j] - x[j] != 0.f)) ? x[j] : 0.f;
            }
    }
    __syncthreads();
    find_not_finite<KIND, D, true>(tile, row0);
    __syncthreads();
}

// Writes a wave's rows: results where the block is in one part, else its sums.
// o[t][i] of lane (r, h) is row r, element 32 t + 8 (i / 4) + 4 h + i % 4; l and lx
// are halves of the row's.
template <int KIND, int D>
BEAM_DEV void write_rows(const AttnPromptArgs& a, const Block& k, const Rows& x, size_t slot, int head, int wave,
                         f32x16 (&o)[D / 32], float m, float l, float lx) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    l = sum_halves(l);
    lx = sum_halves(lx);
    if (k.np > 1) {
        const size_t at = (slot * a.Hkv + head) * kPromptRows + wave * 32 + (lane & 31);
        if (!x.live) return;
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(a.parts + at * D + 32 * t + 2 * i + 4 * h) =
                    make_float4(o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
        if (h == 0) a.ml[at] = make_float4(m, l, lx, 0.f);
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const size_t out = (size_t)(k.first + x.qi) * a.Hq + head * a.G + x.qg;
#pragma unroll
    for (int t = 0; t < D / 32; ++t) {
        if constexpr (KIND == A_F32) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (x.live)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out * D + 32 * t + 2 * i + 4 * h) =
                        make_float4(o[t][i] * inv, o[t][i + 1] * inv, o[t][i + 2] * inv, o[t][i + 3] * inv);
        } else {
            // halves exchange four elements each, so that a lane stores eight in a row
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16x2(o[t][i + 2 * e] * inv, o[t][i + 2 * e + 1] * inv);
                const auto y = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto z = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                if (x.live)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out * D + 32 * t + 2 * i + 8 * h) =
                        make_uint4(y[0], z[0], y[1], z[1]);
            }
        }
    }
    if (a.lse && h == 0 && x.live) a.lse[out] = lx == 0.f ? -INFINITY : m * kLn2 + logf(lx);
}

// Join of a block's parts: a workgroup per (block, key-value head, 256 / (D / 4)
// rows), a row per D/4 lanes; kBatch parts' loads in flight at a time.
template <int KIND, int D>
__global__ __launch_bounds__(256) void beam_attn_prompt_join(AttnPromptArgs a) {
    constexpr int LPR = D / 4, NR = 256 / LPR, PER = kPromptRows / NR, kBatch = 4;
    const int head = blockIdx.x % a.Hkv, at = blockIdx.x / a.Hkv / PER;
    const int rr = blockIdx.x / a.Hkv % PER * NR + threadIdx.x / LPR, d = threadIdx.x % LPR * 4;
    Block k;
    if (a.p.every) {
        const int b = sequence_of(a, at);
        if (!block_of(a, b, at - first_block(a, b), k)) return;
    } else {
        if (!block_of(a, at, 0, k)) return;
    }
    if (k.np <= 1 || k.row0 + rr >= k.row1) return;
    const size_t row = ((size_t)at * a.p.S * a.Hkv + head) * kPromptRows + rr;
    const size_t step = (size_t)a.Hkv * kPromptRows;
    float M = -INFINITY, Ls = 0.f, Lx = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < k.np; s0 += kBatch) {
        float4 v[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const size_t p = row + min(s0 + j, k.np - 1) * step;
            v[j] = a.ml[p];
            o[j] = *reinterpret_cast<const float4*>(a.parts + p * D + d);
        }
        float top = M;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (s0 + j < k.np) top = fmaxf(top, v[j].x);
        const float ts = top == -INFINITY ? 0.f : top;
        const float alpha = __builtin_amdgcn_exp2f(M - ts);
        M = top;
        Ls *= alpha;
        Lx *= alpha;
        O.x *= alpha; O.y *= alpha; O.z *= alpha; O.w *= alpha;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (s0 + j < k.np) {
                const float e = __builtin_amdgcn_exp2f(v[j].x - ts);
                Ls = fmaf(e, v[j].y, Ls);
                Lx = fmaf(e, v[j].z, Lx);
                O.x = fmaf(e, o[j].x, O.x);
                O.y = fmaf(e, o[j].y, O.y);
                O.z = fmaf(e, o[j].z, O.z);
                O.w = fmaf(e, o[j].w, O.w);
            }
    }
    const float inv = Ls == 0.f ? 0.f : 1.0f / Ls;
    const int qi = (k.row0 + rr) / a.G, qg = (k.row0 + rr) % a.G;
    const size_t out = (size_t)(k.first + qi) * a.Hq + head * a.G + qg;
    if constexpr (KIND == A_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out * D + d) =
            make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out * D + d) =
            make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
    if (a.lse && d == 0) a.lse[out] = Lx == 0.f ? -INFINITY : M * kLn2 + logf(Lx);
}

template <int KIND, int D, typename K> hipError_t launch_prompt(K kernel, const AttnPromptArgs& a, hipStream_t st) {
    const unsigned more = a.p.every ? 0 : (unsigned)a.B * (a.p.S - 1);
    const dim3 grid((a.p.blocks + more) * a.Hkv, a.p.every ? a.p.S : 1);
    const hipError_t err = launch(kernel, grid, dim3(256), st, a);
    if (err != hipSuccess || a.p.S == 1) return err;
    constexpr unsigned PER = kPromptRows / (256 / (D / 4));
    return launch(beam_attn_prompt_join<KIND, D>, dim3((a.p.every ? a.p.blocks : (unsigned)a.B) * a.Hkv * PER),
                  dim3(256), st, a);
}

}  // namespace beam
