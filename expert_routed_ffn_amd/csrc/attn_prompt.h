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
BEAM_DEV int first_block_at(const AttnPromptArgs& a, int b, int offset) {
    return (int)((int64_t)offset * a.G / kPromptRows) + b;
}

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
    static constexpr int TILE = KIND == A_F32 || D == 256 ? 32 : 64;
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
        const int lane = threadIdx.x & 63;
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
            const int lane = threadIdx.x & 63;
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

// ---------------------------------------------------------------- the kernel

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

template <int KIND, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void beam_attn_prompt(AttnPromptArgs a) {
    using L = Lds<KIND, D>;
    constexpr int TILE = L::TILE, NT = TILE / 32;    // 32-token blocks of a step
    constexpr int NB = TILE / 16;                    // 16-token blocks of a step
    constexpr int NQ = KIND == A_F32 ? D / 8 : D / 16;   // 16-byte query pieces per lane
    constexpr int ND = D / 32;
    constexpr int ROWS = Stage<KIND, D>::ROWS;
    constexpr bool SC = KIND == A_FP8;
    // two buffers of a step's keys and values, variables of their own: so the
    // compiler sees that reads of one need not wait for loads into the other
    __shared__ __attribute__((aligned(16))) uint8_t sK0[L::BYTES], sV0[L::BYTES], sK1[L::BYTES], sV1[L::BYTES];
    __shared__ __attribute__((aligned(16))) float sKs[2][SC ? TILE : 4], sVs[2][SC ? TILE : 4];
    __shared__ int sBad;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int head = blockIdx.x % a.Hkv, G = a.G;
    const int at = blockIdx.x / a.Hkv;

    // the block and the part: parts 1 .. of the sequences in one block come first,
    // then the blocks, a sequence's last ones, which see most, first
    Block k;
    int part = 0, slot;
    if (a.p.every) {
        const int idx = (int)a.p.blocks - 1 - at;
        const int b = sequence_of(a, idx);
        if (!block_of(a, b, idx - first_block(a, b), k)) return;
        part = blockIdx.y;
        slot = idx * (int)a.p.S + part;
    } else {
        const int extra = a.B * ((int)a.p.S - 1);
        if (at < extra) {
            const int b = at / ((int)a.p.S - 1);
            part = 1 + at % ((int)a.p.S - 1);
            if (!block_of(a, b, 0, k)) return;
        } else {
            const int idx = (int)a.p.blocks - 1 - (at - extra);
            const int b = sequence_of(a, idx);
            if (!block_of(a, b, idx - first_block(a, b), k)) return;
        }
        slot = k.b * (int)a.p.S + part;
    }
    if (part >= k.np) return;
    const int v0 = k.base + part * k.part;
    const int v1 = part + 1 < k.np ? v0 + k.part : k.end;

    // this lane's row and query; rows past the block's last repeat it
    const int row = min(k.row0 + wave * 32 + r, k.row1 - 1);
    const int qi = row / G, qg = row - qi * G;
    const int pos = k.len - k.n + qi;
    const int wlo = k.len - k.n + min(k.row0 + wave * 32, k.row1 - 1) / G;        // the wave's first and last position
    const int whi = k.len - k.n + min(k.row0 + wave * 32 + 31, k.row1 - 1) / G;
    uint4 qf[NQ];
    {
        const size_t off = (size_t)(k.first + qi) * a.qs + (size_t)(head * G + qg) * D;
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + off * L::ES);
#pragma unroll
        for (int c = 0; c < NQ; ++c) qf[c] = q[2 * c + h];
    }

    const float zs = a.scale * kLog2e;
    // reference that the probabilities are relative to, this lane's share of
    // their sum, and (BF) of their sum before they were rounded, which lse needs
    constexpr bool BF = KIND == A_BF16 || KIND == A_FP4;
    float m = -INFINITY, l = 0.f, lx = 0.f;
    f32x16 o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = zeros16();

    // The pages of a step's 16-token blocks, through the scalar cache; they are
    // looked up two steps ahead.  Blocks past the end look up the last one.
    typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
    const scalar_ints table = (scalar_ints)(uintptr_t)(a.table + (size_t)k.b * a.max_pages);
    const auto token = [&](int place) { return place < k.skip ? place : place + k.gap; };   // of a 16-token block
    const int last16 = (v1 - 1) & ~15;
    const auto pages_of = [&](int v, int (&pg)[NB]) {
#pragma unroll
        for (int u = 0; u < NB; ++u) pg[u] = table[token(min(v + 16 * u, last16)) >> a.c.pshift];
    };
    const auto in_cache = [&](int pg) { return (uint32_t)pg < (uint32_t)a.c.n_pages; };

    Stage<KIND, D> ck, cv;
    float ksc = 0.f, vsc = 0.f;
    // the loads of the step at place v, into one of the buffers
    const auto load = [&](int v, const int (&pg)[NB], uint8_t* sK, uint8_t* sV) {
        const int row = wave * ROWS, place = v + (row & ~15);
        int page = 0;
#pragma unroll
        for (int u = 0; u < NB; ++u) page |= pg[u] & -(int)(row / 16 == u);
        const uint8_t *kp, *vp, *kss, *vss;
        kp = vp = kss = vss = reinterpret_cast<const uint8_t*>(kZeros);
        if (place < v1 && in_cache(page)) {
            const size_t at_row = (((size_t)page * a.Hkv + head) << a.c.pshift) +
                                  ((token(place) + (row & 15)) & ((1 << a.c.pshift) - 1));
            kp = static_cast<const uint8_t*>(a.c.k) + at_row * Stage<KIND, D>::CB;
            vp = static_cast<const uint8_t*>(a.c.v) + at_row * Stage<KIND, D>::CB;
            constexpr int SB = KIND == A_FP4 ? D / 32 : 4;   // scale bytes per row
            kss = static_cast<const uint8_t*>(a.c.ks) + at_row * SB;
            vss = static_cast<const uint8_t*>(a.c.vs) + at_row * SB;
        }
        ck.template load<false>(kp, kss, sK, row);
        cv.template load<true>(vp, vss, sV, row);
        if constexpr (SC) {
            ksc = reinterpret_cast<const float*>(kss)[lane % ROWS];
            vsc = reinterpret_cast<const float*>(vss)[lane % ROWS];
        }
    };
    const auto store = [&](uint8_t* sK, uint8_t* sV, int buf) {
        ck.template store<false>(sK, wave * ROWS);
        cv.template store<true>(sV, wave * ROWS);
        if constexpr (SC) {
            if (lane < ROWS) {
                sKs[buf][wave * ROWS + lane] = ksc;
                sVs[buf][wave * ROWS + lane] = vsc;
            }
        }
    };

    if (threadIdx.x == 0) sBad = -1;
    int pg[NB], next[NB];
    if (v0 < v1) {
        pages_of(v0, pg);
        load(v0, pg, sK0, sV0);
        pages_of(v0 + TILE, next);
        store(sK0, sV0, 0);
    }
    // Byte places in LDS of this lane's key piece 2 c + h of row 32 t + r, and of
    // its four value elements for a transposing read: the exchange of pieces is an
    // exclusive or, so piece and block enter by one.
    const int i16 = lane & 15;
    int kat = r * L::RB + L::kslot(r, h) * 16;                    // ^ 32 c, + 32 t RB
    int vat = (4 * h + i16 / 4) * L::RB +
              L::vslot(4 * h + i16 / 4, (lane & 16) / 8 + i16 % 4 / 2) * 16 + i16 % 2 * 8;   // ^ (64 t + 32 y), + (16 s + 8 y) RB
    // one step: buffer `buf` (sK, sV) is worked on while the other (oK, oV) fills
    const auto step = [&](int v, int buf, uint8_t* sK, uint8_t* sV, uint8_t* oK, uint8_t* oV) {
        __builtin_amdgcn_s_waitcnt(0);   // this wave's loads to LDS have landed
        __syncthreads();                 // everyone's, and no one reads the other buffer any more
        const bool more = v + TILE < v1;
        // whether every row of the block, and of the wave, sees all of the step's tokens
        const int t0 = token(v), t1 = t0 + TILE - 1;
        bool ok = v + TILE <= v1 && (v >= k.skip || v + TILE <= k.skip);
#pragma unroll
        for (int u = 0; u < NB; ++u) ok = ok && in_cache(pg[u]);
        const bool all = ok && t1 <= k.p0 && (a.window == 0 || t0 > k.p1 - a.window || t1 < a.sinks);
        const bool mine = ok && t1 <= wlo && (a.window == 0 || t0 > whi - a.window || t1 < a.sinks);
        uint32_t there = 0;              // 16-token blocks that there are
#pragma unroll
        for (int u = 0; u < NB; ++u) there |= v + 16 * u < v1 && in_cache(pg[u]) ? 1u << u : 0u;
        if (more) {
            load(v + TILE, next, oK, oV);
#pragma unroll
            for (int u = 0; u < NB; ++u) pg[u] = next[u];
            pages_of(v + 2 * TILE, next);
        }
        const auto sees = [&](int u, int x) {   // whether this lane's row sees token x of the step's 16-token block u
            const int tok = token(v + 16 * u) + x;
            return (there >> u & 1) && tok <= pos && (a.window == 0 || tok > pos - a.window || tok < a.sinks);
        };
        // A value that is not finite must not reach rows that do not see it: 0
        // times it is NaN.  Where rows differ in what they see, the step's values
        // are looked through first.  If one is not finite, it is added to the
        // rows that see it, with any weight, and is 0 in LDS from there on.
        if (!all) {
            const auto mend = [&](bool set) {
                bool bad = false;
                uint8_t* p = sV + wave * ROWS * L::RB;
                for (int i = lane; i < ROWS * L::NP; i += 64) {
                    uint4* w = reinterpret_cast<uint4*>(p + i * 16);
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
                    if (set && here) *w = make_uint4(x[0], x[1], x[2], x[3]);
                    bad |= here;
                }
                return bad;
            };
            if (__any(mend(false)) && lane == 0) sBad = v;
            __syncthreads();
            if (sBad == v) {
#pragma unroll 1
                for (int y = 0; y < TILE; ++y) {
                    const bool add = sees(y / 16, y % 16);
#pragma unroll
                    for (int t = 0; t < ND; ++t)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const int e = 32 * t + 2 * i + 4 * h;
                            const uint8_t* w = sV + y * L::RB + L::vslot(y, e * L::ES / 16) * 16 + e * L::ES % 16;
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
                mend(true);
                __syncthreads();
            }
        }

        // the registers that 256 elements leave hold no sixteen places
        if constexpr (D == 256) asm volatile("" : "+v"(kat), "+v"(vat));

        // scores: lane (r, h) gets row r, tokens 32 t + 8 (i / 4) + 4 h + i % 4
        f32x16 z[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            z[t] = zeros16();
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                const uint4 kf = *reinterpret_cast<const uint4*>(sK + (kat ^ (32 * c)) + 32 * t * L::RB);
                if constexpr (KIND == A_F32) {
                    const uint32_t kw[4] = {kf.x, kf.y, kf.z, kf.w}, qw[4] = {qf[c].x, qf[c].y, qf[c].z, qf[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kw[e]), __uint_as_float(qw[e]), z[t],
                                                                    0, 0, 0);
                } else {
                    z[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf),
                                                                   __builtin_bit_cast(bf16x8, qf[c]), z[t], 0, 0, 0);
                }
            }
            if constexpr (SC) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&sKs[buf][32 * t + 2 * i + 4 * h]);
                    z[t][i] *= f.x; z[t][i + 1] *= f.y; z[t][i + 2] *= f.z; z[t][i + 3] *= f.w;
                }
            }
        }
        if (!mine) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    z[t][i] = sees(2 * t + i / 8, 8 * (i / 4 % 2) + 4 * h + i % 4) ? z[t][i] : -INFINITY;
        }
        // The reference moves (and what was summed is rescaled) only when a
        // score exceeds it by 8 powers of two.
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, z[t][i]);
        top *= zs;
        if (__any(top > m + 8.f)) {
            const float mn = fmaxf(m, max_halves(top));
            const float alpha = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            l *= alpha;
            lx *= alpha;
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[t][i] *= alpha;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        uint32_t pb[KIND == A_F32 ? 1 : NT * 8];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[t][i] = __builtin_amdgcn_exp2f(fmaf(z[t][i], zs, -ms));
            if (!BF || a.lse) {
                float& sum = BF ? lx : l;
#pragma unroll
                for (int i = 0; i < 16; i += 4) sum += (z[t][i] + z[t][i + 1]) + (z[t][i + 2] + z[t][i + 3]);
            }
            if constexpr (KIND != A_F32) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    float y[4] = {z[t][i], z[t][i + 1], z[t][i + 2], z[t][i + 3]};
                    if constexpr (SC) {
                        const float4 f = *reinterpret_cast<const float4*>(&sVs[buf][32 * t + 2 * i + 4 * h]);
                        y[0] *= f.x; y[1] *= f.y; y[2] *= f.z; y[3] *= f.w;
                        if (!mine) {   // a scale that is not finite, of a token that is not seen
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = z[t][i + e] == 0.f ? 0.f : y[e];
                        }
                    }
                    pb[8 * t + i / 2] = pack_bf16x2(y[0], y[1]);
                    pb[8 * t + i / 2 + 1] = pack_bf16x2(y[2], y[3]);
                    if constexpr (BF) {
                        // summed as they enter the product, so that their rounding
                        // cancels: equal values come back as themselves
                        typedef __bf16 pair __attribute__((ext_vector_type(2)));
                        const pair one = {(__bf16)1.f, (__bf16)1.f};
                        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair, pb[8 * t + i / 2]), one, l, false);
                        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair, pb[8 * t + i / 2 + 1]), one, l, false);
                    }
                }
            }
        }

        // values: V^T fragments of 32 elements by 16 tokens
        const auto vfrag = [&](int t, int s) {   // elements 32 t + lane % 32, tokens 16 s + 8 (j / 4) + 4 h + j % 4
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            uint4 f;
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                // the 16 lanes of a group read four rows of 16 elements, lane i row
                // i / 4 and elements 4 (i % 4) .. + 3, and get element i of each
                const uint8_t* p = sV + (vat ^ (64 * t + 32 * y)) + (16 * s + 8 * y) * L::RB;
                const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                              (__attribute__((address_space(3))) s16x4*)p));
                w[2 * y] = x.x;
                w[2 * y + 1] = x.y;
            }
            f = make_uint4(w[0], w[1], w[2], w[3]);
            return f;
        };
        const auto vword = [&](int t, int i) {   // fp32: element 32 t + lane % 32 of token 8 (i / 4) + 4 h + i % 4
            const int vr = 8 * (i / 4) + 4 * h + i % 4, e = 32 * t + r;
            return *reinterpret_cast<const float*>(sV + vr * L::RB + L::vslot(vr, e / 4) * 16 + (e % 4) * 4);
        };
#pragma unroll
        for (int t = 0; t < ND; ++t) {
            if constexpr (KIND == A_F32) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(vword(t, i), z[0][i], o[t], 0, 0, 0);
            } else {
#pragma unroll
                for (int s = 0; s < NB; ++s)
                    o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, vfrag(t, s)),
                        __builtin_bit_cast(bf16x8, make_uint4(pb[4 * s], pb[4 * s + 1], pb[4 * s + 2], pb[4 * s + 3])),
                        o[t], 0, 0, 0);
            }
        }
        if (more) store(oK, oV, buf ^ 1);
    };
    for (int v = v0; v < v1; v += 2 * TILE) {
        step(v, 0, sK0, sV0, sK1, sV1);
        if (v + TILE < v1) step(v + TILE, 1, sK1, sV1, sK0, sV0);
    }

    // o[t][i] of lane (r, h) is row r, element 32 t + 8 (i / 4) + 4 h + i % 4
    l = sum_halves(l);
    lx = BF ? sum_halves(lx) : l;
    const int my = k.row0 + wave * 32 + r;
    if (k.np > 1) {
        const size_t at_row = ((size_t)slot * a.Hkv + head) * kPromptRows + wave * 32 + r;
        if (my < k.row1) {
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(a.parts + at_row * D + 32 * t + 2 * i + 4 * h) =
                        make_float4(o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
            if (h == 0) a.ml[at_row] = make_float4(m, l, lx, 0.f);
        }
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const size_t out = ((size_t)(k.first + qi) * a.Hq + head * G + qg);
    if constexpr (KIND == A_F32) {
        if (my < k.row1) {
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out * D + 32 * t + 2 * i + 4 * h) =
                        make_float4(o[t][i] * inv, o[t][i + 1] * inv, o[t][i + 2] * inv, o[t][i + 3] * inv);
        }
    } else {
        // halves exchange four elements each, so that a lane stores eight in a row
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16x2(o[t][i + 2 * e] * inv, o[t][i + 2 * e + 1] * inv);
                const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                if (my < k.row1)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out * D + 32 * t + 2 * i + 8 * h) =
                        make_uint4(x[0], y[0], x[1], y[1]);
            }
    }
    if (a.lse && h == 0 && my < k.row1) a.lse[out] = lx == 0.f ? -INFINITY : m * kLn2 + logf(lx);
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

template <int KIND, int D> static hipError_t launch_prompt(const AttnPromptArgs& a, hipStream_t st) {
    const unsigned more = a.p.every ? 0 : (unsigned)a.B * (a.p.S - 1);
    const dim3 grid((a.p.blocks + more) * a.Hkv, a.p.every ? a.p.S : 1);
    const hipError_t err = launch(beam_attn_prompt<KIND, D>, grid, dim3(256), st, a);
    if (err != hipSuccess || a.p.S == 1) return err;
    constexpr unsigned PER = kPromptRows / (256 / (D / 4));
    return launch(beam_attn_prompt_join<KIND, D>, dim3((a.p.every ? a.p.blocks : (unsigned)a.B) * a.Hkv * PER),
                  dim3(256), st, a);
}

template <int KIND> static hipError_t launch_prompt_d(const AttnPromptArgs& a, hipStream_t st) {
    if (a.D == 64) return launch_prompt<KIND, 64>(a, st);
    if (a.D == 128) return launch_prompt<KIND, 128>(a, st);
    return launch_prompt<KIND, 256>(a, st);
}

}  // namespace beam
