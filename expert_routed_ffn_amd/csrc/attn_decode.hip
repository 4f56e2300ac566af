// Attention of one new token per sequence over a paged key-value cache.
//
// For each (sequence, key-value head) the G = Hq/Hkv query heads form the
// columns of two matrix products over the cached tokens,
//   Z^T [tokens, G] = K Q^T     and     O^T [D, G] = V^T P^T,
// with one pass over the cache and the running maximum and sum of the
// softmax beside them.  Everything stays in registers: the first product's
// result layout (lane (r, g) holds query column r and tokens 4g..4g+3 of a
// 16-token block) is the layout of the second product's right operand when
// the reduction index (g, 4u + i) stands for token 16u + 4g + i of a
// 32-token tile, so the probabilities move between no lanes, and lane
// (r, g) reads the same tokens' value elements r * D/16 .. + D/16 - 1 as whole
// row pieces; output block t then holds rows d = r * D/16 + t.
//
// The cache's length is split over workgroups (parts) and over the four waves
// of a workgroup (tiles in turn).  The waves' results are joined through LDS,
// the parts' through the workspace by a second kernel; a batch of more parts
// than the grid holds for each sequence has them listed by one before.
//
// HBM bounds it: 2 flops per byte and query at most (e4m3) are far below what
// the matrix cores give, with the padding of G to 16 columns and the second
// product's two operands too.  64 sequences of 8192 tokens, 48 heads over 8 of
// 128: bf16 340 us, 6.3 TB/s; e4m3 181 us, 6.1 TB/s; fp32 670 us, 6.4 TB/s; one
// sequence of 131071, bf16: 87 us, 6.1 TB/s (a read-only stream on this card
// reaches 6.3 with plain loads, 7.0 with non-temporal ones; a copy 4.7).  Small
// calls are latency: 8 sequences of up to 2048 tokens take 9 us for a chain of
// length, page, two steps of keys and values, join, store, and 3 us to join
// their parts.
#include "common.h"
#include "kernels.h"

namespace beam {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Tokens per wave step, by cache element.
template <int KIND> constexpr int tile_tokens() { return KIND == A_F32 ? 16 : 32; }

// Parts of a sequence, chosen on the device from its own length: `want` even
// ones, of kMinPart to kMaxPart tokens; `want` is what gives kWantWG workgroups
// in all.  Two workgroups per CU keep the memory busy, and a sequence in one
// part needs no join (64 sequences, window 512, e4m3: 13.5 us in one part, 19.3
// in two).  Parts are bounded so that a batch of very different lengths still
// spreads over the chip (1 .. 32768 tokens, e4m3: 302, 292, 288 and 304 us for
// parts of up to 1024, 2048, 4096 and 8192 tokens) until the sequences alone
// do that, and even because a power of two leaves a small batch of different
// lengths with few, long ones (8 of 94 .. 5985, bf16: 28.5 -> 23.9 us).
//
// S, the most parts a sequence of max_len tokens can have, sizes grid and
// workspace while there are at most kMostWG workgroups; parts are numbered
// outermost, so that those which a short sequence lacks come last and only
// end (64 sequences of 2048 tokens, e4m3: 43.6 us where 2048 are expected; 120
// us numbered innermost with kMostWG = 16384).
//
// Where that bound would make parts longer than kMaxPart, they are listed by a
// kernel of one workgroup first (beam_attn_list): the grid holds `want` parts of
// every sequence and kMostWG workgroups (`extra` parts of each head) more,
// wherever they are needed, and parts grow beyond kMaxPart, to the same multiple
// for all sequences, only where the lengths together ask for more.  Cut to S
// parts instead, one long sequence among many runs on its own (e4m3, 131072
// tokens beside 300 sequences of 512: 1061 us, listed 108; beside 1000: 1181 and
// 250; 256 sequences of 1 .. 32768: 981 and 963), while without long ones the list
// is 2 to 4 % (64 sequences of 2048, 131072 expected: 46.3 us and 48.2; 2000 of
// 512: 363 and 376) and at worst its launch (64 of 512: 18.3 and 19.7).  From
// kMostListed sequences on there are workgroups enough without parts, and each
// is one: a long one among them ends by itself.
constexpr int kWantWG = 512, kMostWG = 4096, kMinPart = 256, kMaxPart = 4096, kRound = 128, kMostListed = 4096;
AttnSplit attn_decode_split(int B, int Hkv, int max_len, int window) {
    // a window's tokens begin inside a 16-token block
    const int64_t span = window > 0 && window < max_len ? (int64_t)window + 15 : max_len;
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

// The tokens that a sequence's query sees, [start, len), cut into n parts of
// `part` tokens (whole workgroup steps) from `base` on: of at most `scale` times
// kMaxPart tokens if listed, else into no more than S where the sequence is longer
// than expected.
struct Span {
    int start, len, base, part, n;
};
BEAM_DEV int table_tokens(const AttnDecodeArgs& a) {
    return (int)min((int64_t)a.max_pages << a.c.pshift, (int64_t)kMaxLen);
}
BEAM_DEV void see(const AttnDecodeArgs& a, int len, Span& p) {
    p.len = len;
    p.start = a.window > 0 ? max(0, len - a.window) : 0;
    p.base = p.start & ~15;
}
template <bool LISTED> BEAM_DEV Span span_of(const AttnDecodeArgs& a, int cap, int len, uint32_t scale = 1) {
    Span p;
    see(a, min(max(len, 0), cap), p);
    const uint32_t all = (uint32_t)(p.len - p.base);
    uint32_t part = (all + a.p.want - 1) / a.p.want;
    part = min(max(part, (uint32_t)kMinPart), (uint32_t)kMaxPart * scale);
    if (!LISTED && (uint64_t)part * a.p.S < all) part = (all + a.p.S - 1) / a.p.S;
    part = (part + kRound - 1) & ~(uint32_t)(kRound - 1);
    p.part = (int)part;
    p.n = (int)((all + part - 1) / part);
    return p;
}

// The list of all parts: those of the sequences in several parts, which take
// longest, then the sequences in one (or without tokens).  Each has its sequence,
// its number there, the sequence's length and the tokens per part; -1 stands
// behind the last.  For the join: the sequences in several parts, their first
// part and how many.  The lengths are summed in units of kMaxPart, which gives the
// scale of the parts: with U units in all and scale m = ceil(U / extra), a
// sequence of u units has at most want + u / m parts, so there are no more than
// rows = B * want + extra.  One workgroup; the launch and its work take 3 to 5 us.
constexpr int kListThreads = 1024;
__global__ __launch_bounds__(kListThreads) void beam_attn_list(AttnDecodeArgs a) {
    constexpr int kPer = kMostListed / kListThreads;
    const int per = (a.B + kListThreads - 1) / kListThreads;   // neighbouring sequences of a thread
    __shared__ int at[kMostListed], seq[kMostListed], sums[kListThreads / 64];
    const int cap = table_tokens(a), tid = threadIdx.x;
    const auto scan = [&](int v, int* total) {         // exclusive sum over the workgroup
        int incl = v;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(incl, o, kWave);
            if ((tid & 63) >= o) incl += u;
        }
        __syncthreads();
        if ((tid & 63) == 63) sums[tid >> 6] = incl;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kListThreads / 64; ++i) {
            before += i < (tid >> 6) ? sums[i] : 0;
            all += sums[i];
        }
        *total = all;
        return before + incl - v;
    };
    int len[kPer], units = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= per) break;
        const int b = tid * per + i;
        len[i] = b < a.B ? a.lens[b] : 0;
        const Span p = span_of<true>(a, cap, len[i]);
        units += (p.len - p.base + kMaxPart - 1) / kMaxPart;   // 2^18 at most, of 2^12 sequences
    }
    scan(units, &total);
    const uint32_t scale = max(1u, min(((uint32_t)total + a.p.extra - 1) / a.p.extra, (uint32_t)(kMaxLen / kMaxPart)));

    // sequences in several parts, and their parts in the upper bits: fewer than 2^12 and 2^13
    int n[kPer], many = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= per) break;
        n[i] = span_of<true>(a, cap, len[i], scale).n;
        if (n[i] > 1) many += (n[i] << 12) + 1;
    }
    int before = scan(many, &total);
    const int parts = total >> 12, cut = total & 0xFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        if (i >= per || b >= a.B) break;
        const int k = before & 0xFFF, first = before >> 12;
        if (n[i] > 1) {
            at[k] = first;
            seq[k] = b;
            a.lists[k] = make_int4(b, first, n[i], 0);
            before += (n[i] << 12) + 1;
        } else {
            const Span p = span_of<true>(a, cap, len[i], scale);
            a.items[parts + b - k] = make_int4(b, 0, p.len, p.part);
        }
    }
    __syncthreads();
    for (int i = tid; i < (int)a.p.rows; i += kListThreads) {
        if (i < parts) {
            int lo = 0, hi = cut;                      // at[lo] <= i < at[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (at[mid] <= i) lo = mid;
                else hi = mid;
            }
            const Span p = span_of<true>(a, cap, a.lens[seq[lo]], scale);
            a.items[i] = make_int4(seq[lo], i - at[lo], p.len, p.part);
        } else if (i >= parts + a.B - cut) {
            a.items[i] = make_int4(-1, 0, 0, 0);
        }
    }
    for (int i = cut + tid; i < (int)a.p.joins; i += kListThreads) a.lists[i] = make_int4(-1, 0, 0, 0);
}

// four e4m3 codes to bf16 (exact): codes 0, 1 and codes 2, 3
BEAM_DEV uint32_t e4m3_lo(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
}
BEAM_DEV uint32_t e4m3_hi(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
}

// NW 32-bit words from global memory (16-, 8- or 4-byte pieces).  STREAM: as
// non-temporal loads.
template <int NW, bool STREAM = false> BEAM_DEV void ldw(const void* p, uint32_t (&w)[NW]) {
    constexpr int PW = NW % 4 == 0 ? 4 : NW;   // words per load
    typedef uint32_t piece __attribute__((ext_vector_type(PW)));
    static_assert(NW % PW == 0 && (PW == 4 || PW == 2 || PW == 1), "");
#pragma unroll
    for (int i = 0; i < NW / PW; ++i) {
        const piece* q = static_cast<const piece*>(p) + i;
        piece v;
        if constexpr (STREAM) v = __builtin_nontemporal_load(q);
        else v = *q;
#pragma unroll
        for (int j = 0; j < PW; ++j) w[PW * i + j] = v[j];
    }
}

BEAM_DEV f32x4 mfma_bf16(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, make_uint4(a0, a1, a2, a3)),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight weights as the sum of two bf16 operands: the leading 8 bits, and what
// is left of each, rounded, so that a weight is off by 2^-15 at most.  One
// rounded operand does not cancel against the softmax's sum, so that equal
// values came back as their neighbours.  Most of the second product hides behind
// HBM (e4m3, one sequence of 131071: 45.1 us with and without; 64 of 8192: 179 ->
// 181; 64 windows of 512: 13.1 -> 13.4), least where 64 queries share a head (64
// sequences of 8192: e4m3 47 -> 52, bf16 61 -> 64).  The 2^-24 of the weight
// keep the rest from being zero, which times an infinite value would be NaN.
BEAM_DEV void split_bf16(const float (&y)[8], uint4& hi, uint4& lo) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = fmaf(y[i], 0x1p-24f, y[i] - __uint_as_float(__float_as_uint(y[i]) & 0xFFFF0000u));
    }
    const auto top = [&](int i) {
        return __builtin_amdgcn_perm(__float_as_uint(y[i + 1]), __float_as_uint(y[i]), 0x07060302u);
    };
    hi = make_uint4(top(0), top(2), top(4), top(6));
    lo = make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
}

// Transposes 16-byte pieces among groups of N = 2 or 4 neighbouring lanes:
// lane n's piece i becomes lane i's piece n.
template <int CTRL> BEAM_DEV uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int N> BEAM_DEV void lane_transpose(uint32_t (*w)[4]) {
    constexpr int kXor1 = 0xB1, kXor2 = 0x4E;   // exchange with the lane 1 or 2 away
    const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
    if constexpr (N >= 2) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[i][e], b = w[i + 1][e];
                const uint32_t xa = dpp<kXor1>(a), xb = dpp<kXor1>(b);   // every lane takes part
                w[i][e] = odd ? xb : a;
                w[i + 1][e] = odd ? b : xa;
            }
    }
    if constexpr (N == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[i][e], b = w[i + 2][e];
                const uint32_t xa = dpp<kXor2>(a), xb = dpp<kXor2>(b);
                w[i][e] = upper ? xb : a;
                w[i + 2][e] = upper ? b : xa;
            }
    }
}

// maximum over the four lanes (r, 0..3) that hold a query's tokens
BEAM_DEV float max_over_g(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
BEAM_DEV float sum_over_g(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// A wave's state over the tokens it has seen: 16 * QT queries.
//   m   reference that the probabilities are relative to (2^(z - m)); -inf
//       before the first score
//   l   this lane's share of the sum of probabilities
//   o   weighted sum of values
template <int D, int QT> struct Acc {
    float m[QT], l[QT];
    f32x4 o[QT][D / 16];
};

// With 32 queries a wave, or heads of 256, the registers are held to two waves
// per SIMD (64 queries on one head, e4m3: 61 -> 52 us; D = 256, 253 windows of 128,
// e4m3: 51 -> 32 us); fp32 would spill there (129 -> 146 us), and else what the
// compiler takes is best.
template <int KIND, int D, int QT, bool LISTED>
__global__ __launch_bounds__(256, KIND != A_F32 && (QT == 2 || D == 256) ? 2 : 1) void beam_attn_decode(AttnDecodeArgs a,
                                                                                         int qgroups) {
    constexpr int TILE = tile_tokens<KIND>(), NU = TILE / 16;   // 16-token blocks per step
    constexpr int STEP = 4 * TILE;                              // tokens per workgroup step
    constexpr int ES = KIND == A_F32 ? 4 : (KIND == A_BF16 ? 2 : 1);   // bytes per cache element
    constexpr int DL = D / 16;                                  // value elements per lane and token
    constexpr int NK = KIND == A_F32 ? D / 16 : D / 32;         // key fragments per token
    constexpr int KW = KIND == A_FP8 ? 2 : 4;                   // words per key fragment
    constexpr int NC = NK * KW / 4;                             // 16-byte key pieces per lane and token
    // pieces exchanged among NT lanes (see the key loads)
    constexpr int NT = KIND == A_F32 || (KIND == A_BF16 && QT == 1) ? 1 : (NC < 4 ? NC : 4);
    constexpr int PF = 4 / KW;                                  // fragments per piece
    constexpr int KE = 4 * KW / ES;                             // elements per key fragment
    constexpr int VW = DL * ES / 4;                             // words per lane and value row
    __shared__ float sO[4][16][D + 4];
    __shared__ float sM[4][16], sL[4][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    // Grid: (sequence, head) along x, parts along y; (part, head) along x where
    // parts are listed.  Workgroups that differ in their query rows only follow
    // each other on one XCD, so that its L2 serves the keys and values of all
    // but the first.
    int bh = blockIdx.x, qg = 0;
    if (qgroups > 1) {
        const int j = bh >> 3;
        qg = j % qgroups;
        bh = j / qgroups * 8 + (bh & 7);
    }
    const int h = bh % a.Hkv, G = a.G;
    int b = bh / a.Hkv, s = blockIdx.y;           // listed: the part's number in place of b
    Span sp;
    const size_t prow = LISTED ? b : (size_t)b * a.p.S + s;   // the part's row in the workspace
    if (b >= (LISTED ? (int)a.p.rows : a.B)) return;
    if constexpr (LISTED) {
        const int4 item = a.items[b];
        if (item.x < 0) return;
        b = item.x;
        s = item.y;
        see(a, item.z, sp);
        sp.part = item.w;
        sp.n = (int)((uint32_t)(sp.len - sp.base + sp.part - 1) / (uint32_t)sp.part);
    } else {
        sp = span_of<false>(a, table_tokens(a), a.lens[b]);
    }
    if (s > 0 && s >= sp.n) return;               // no tokens; part 0 of an empty row goes on
    const int t0 = sp.base + s * sp.part;
    const int t1 = s + 1 < sp.n ? t0 + sp.part : sp.len;

    // query fragments: lane (r, g) holds column r of each 16-query block; the
    // reduction index (g, c, j) stands for the key element that lane g's
    // fragment c holds in place j: its quarter of the row in order (NT > 1), or
    // every fourth piece
    uint32_t qf[QT][NK][4];
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        const int qrow = (qg * QT + j) * 16 + r;
        const size_t qoff = (size_t)b * a.qs + (size_t)(h * G + min(qrow, G - 1)) * D;
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const int e = KE * (NT > 1 ? NK * g + c : (c / PF * 4 + g) * PF + c % PF);
            if constexpr (KIND == A_F32) ldw<4>(static_cast<const float*>(a.q) + qoff + e, qf[j][c]);
            else ldw<4>(static_cast<const uint16_t*>(a.q) + qoff + e, qf[j][c]);
        }
    }

    Acc<D, QT> acc;
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        acc.m[j] = -INFINITY;
        acc.l[j] = 0.f;
#pragma unroll
        for (int t = 0; t < DL; ++t) acc.o[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const float zs = a.scale * kLog2e;
    const int pmask = (1 << a.c.pshift) - 1;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    const uint8_t* kc = static_cast<const uint8_t*>(a.c.k);
    const uint8_t* vc = static_cast<const uint8_t*>(a.c.v);

    // pages of a step's 16-token blocks (-1 past the end); they are read one
    // step ahead of the keys and values
    auto pages_of = [&](int tile, int (&pg)[NU]) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int tok = tile + 16 * u;
            pg[u] = tok < t1 ? table[tok >> a.c.pshift] : -1;
        }
    };
    int pg[NU];
    int tile = t0 + wave * TILE;
    pages_of(tile, pg);

    for (; tile < t1; tile += STEP) {
        // all of the step's loads, before any use: a block past the end or
        // on a bad page reads page 0 and is masked below
        size_t row[NU];
        bool ok[NU];
        bool full = tile >= sp.start && tile + TILE <= t1;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            ok[u] = (uint32_t)pg[u] < (uint32_t)a.c.n_pages;
            full = full && ok[u];
            row[u] = (((size_t)(ok[u] ? pg[u] : 0) * a.Hkv + h) << a.c.pshift) + ((tile + 16 * u) & pmask);
        }
        uint32_t kw[NU][NC][4], vw[NU][4][VW];
        float4 ks[NU], vs[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            // The cache unit takes four lanes at a time, in pieces that adjoin.
            // NT = 1: the lanes of a row are 16 apart, and each reads 16 bytes
            // of its row on its own.  NT > 1: neighbouring lanes read one row's
            // pieces side by side, the lowest lane's row, then the next one's,
            // and exchange them below.  That pays where those accesses bound
            // the kernel: at one byte an element (64 sequences of 8192: 234 ->
            // 217 us) and where several workgroups read the same keys (64
            // queries on one head, bf16: 68 -> 63 us); elsewhere HBM bounds it
            // and the exchange costs a percent.
            const uint8_t* kr = kc + (row[u] + (r & ~(NT - 1))) * (D * ES) +
                                (NT > 1 ? g * (D * ES / 4) + (r & (NT - 1)) * 16 : g * 16);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                ldw<4>(kr + (NT > 1 ? (c % NT) * (D * ES) + (c / NT) * (NT * 16) : c * 64), kw[u][c]);
            if constexpr (KIND == A_FP8) ks[u] = *reinterpret_cast<const float4*>(a.c.ks + row[u] + 4 * g);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            // streamed: whole cache lines of a wave's load, read by no one else
            // while they matter (64 sequences of 8192 tokens: bf16 391 -> 356 us,
            // e4m3 217 -> 203 us; the keys too: 358 and 197 us, but a quarter
            // slower where two waves read the same keys or the lines are split)
            const uint8_t* vr = vc + (row[u] + 4 * g) * (D * ES) + r * (VW * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) ldw<VW, true>(vr + i * (D * ES), vw[u][i]);
            if constexpr (KIND == A_FP8) vs[u] = *reinterpret_cast<const float4*>(a.c.vs + row[u] + 4 * g);
        }
        pages_of(tile + STEP, pg);
        __builtin_amdgcn_sched_barrier(0);

        // scores in powers of two; lane (r, g): query r, tokens 16u + 4g + i
        float p[QT][NU][4];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if constexpr (NT > 1) {
#pragma unroll
                for (int c = 0; c < NC; c += NT) lane_transpose<NT>(&kw[u][c]);   // to each lane its own row
            }
            const auto key = [&](int c, int e) { return kw[u][(c * KW + e) / 4][(c * KW + e) % 4]; };
            f32x4 z[QT];
#pragma unroll
            for (int j = 0; j < QT; ++j) z[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                if constexpr (KIND == A_F32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < QT; ++j)
                            z[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __uint_as_float(key(c, e)), __uint_as_float(qf[j][c][e]), z[j], 0, 0, 0);
                } else {
                    uint32_t w[4];
                    if constexpr (KIND == A_BF16) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = key(c, e);
                    } else {
                        w[0] = e4m3_lo(key(c, 0));
                        w[1] = e4m3_hi(key(c, 0));
                        w[2] = e4m3_lo(key(c, 1));
                        w[3] = e4m3_hi(key(c, 1));
                    }
#pragma unroll
                    for (int j = 0; j < QT; ++j)
                        z[j] = mfma_bf16(w[0], w[1], w[2], w[3],
                                         make_uint4(qf[j][c][0], qf[j][c][1], qf[j][c][2], qf[j][c][3]), z[j]);
                }
            }
            float f[4] = {zs, zs, zs, zs};
            if constexpr (KIND == A_FP8) {
                f[0] *= ks[u].x; f[1] *= ks[u].y; f[2] *= ks[u].z; f[3] *= ks[u].w;
            }
#pragma unroll
            for (int j = 0; j < QT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[j][u][i] = z[j][i] * f[i];
        }
        if (!full) {
            // scores of tokens that are not seen leave nothing, and their
            // values, which may be anything, count as zeros
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = tile + 16 * u + 4 * g + i;
                    const bool live = ok[u] && tok >= sp.start && tok < t1;
#pragma unroll
                    for (int j = 0; j < QT; ++j) p[j][u][i] = live ? p[j][u][i] : -INFINITY;
#pragma unroll
                    for (int w = 0; w < VW; ++w) vw[u][i][w] = live ? vw[u][i][w] : 0u;
                    if constexpr (KIND == A_FP8) {
                        float* v4 = reinterpret_cast<float*>(&vs[u]);
                        v4[i] = live ? v4[i] : 0.f;
                    }
                }
        }
#pragma unroll
        for (int j = 0; j < QT; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, p[j][u][i]);
            // the reference moves (and what was summed is rescaled) only
            // when a score exceeds it by kSlack powers of two: probabilities
            // up to 2^kSlack lose nothing in fp32 sums or bf16 operands
            constexpr float kSlack = 8.f;
            if (__any(top > acc.m[j] + kSlack)) {
                const float mn = fmaxf(acc.m[j], max_over_g(top));
                const float alpha = __builtin_amdgcn_exp2f(acc.m[j] - (mn == -INFINITY ? 0.f : mn));
                acc.m[j] = mn;
                acc.l[j] *= alpha;
#pragma unroll
                for (int t = 0; t < DL; ++t) acc.o[j][t] *= alpha;
            }
            const float ms = acc.m[j] == -INFINITY ? 0.f : acc.m[j];
            float ps = 0.f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[j][u][i] = __builtin_amdgcn_exp2f(p[j][u][i] - ms);   // unseen: exp2(-inf) = 0
                    ps += p[j][u][i];
                }
            acc.l[j] += ps;
        }

        if constexpr (KIND == A_F32) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < DL; ++t)
#pragma unroll
                        for (int j = 0; j < QT; ++j)
                            acc.o[j][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __uint_as_float(vw[u][i][t]), p[j][u][i], acc.o[j][t], 0, 0, 0);
        } else {
            // 32 tokens at a time: blocks u and u + 1
#pragma unroll
            for (int u = 0; u < NU; u += 2) {
                uint4 ph[QT], pl[QT];
#pragma unroll
                for (int j = 0; j < QT; ++j) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = p[j][u][i];
                        y[4 + i] = p[j][u + 1][i];
                    }
                    if constexpr (KIND == A_FP8) {   // the value row's scale
                        y[0] *= vs[u].x; y[1] *= vs[u].y; y[2] *= vs[u].z; y[3] *= vs[u].w;
                        y[4] *= vs[u + 1].x; y[5] *= vs[u + 1].y; y[6] *= vs[u + 1].z; y[7] *= vs[u + 1].w;
                    }
                    split_bf16(y, ph[j], pl[j]);
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    // tokens 2n, 2n + 1 of element t side by side
                    constexpr int TW = 4 / ES;   // elements per word
                    uint32_t av[TW][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t x0 = vw[u + n / 2][2 * (n % 2)][w], x1 = vw[u + n / 2][2 * (n % 2) + 1][w];
                        if constexpr (KIND == A_BF16) {
                            av[0][n] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                            av[1][n] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                        } else {
                            const uint32_t y0 = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                            const uint32_t y1 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                            av[0][n] = e4m3_lo(y0);
                            av[1][n] = e4m3_hi(y0);
                            av[TW - 2][n] = e4m3_lo(y1);
                            av[TW - 1][n] = e4m3_hi(y1);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < TW; ++e)
#pragma unroll
                        for (int j = 0; j < QT; ++j)
                            acc.o[j][w * TW + e] =
                                mfma_bf16(av[e][0], av[e][1], av[e][2], av[e][3], ph[j], acc.o[j][w * TW + e]);
#pragma unroll
                    for (int e = 0; e < TW; ++e)
#pragma unroll
                        for (int j = 0; j < QT; ++j)
                            acc.o[j][w * TW + e] =
                                mfma_bf16(av[e][0], av[e][1], av[e][2], av[e][3], pl[j], acc.o[j][w * TW + e]);
                }
            }
        }
    }

    // join the four waves, 16 queries at a time: o[t][i] of lane (r, g) is
    // query r, d = (4g + i) * DL + t
    const bool whole = sp.n <= 1;                 // the only part: no join to come
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        const int q0 = (qg * QT + j) * 16;
        if (q0 >= G) break;
        if (j > 0) __syncthreads();
        const float l = sum_over_g(acc.l[j]);
        if (g == 0) {
            sM[wave][r] = acc.m[j];
            sL[wave][r] = l;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < DL; ++t) sO[wave][r][(4 * g + i) * DL + t] = acc.o[j][t][i];
        __syncthreads();
        const int rows = min(16, G - q0);
        for (int y = threadIdx.x; y < rows * (D / 4); y += 256) {
            const int q = y / (D / 4), d = y % (D / 4) * 4;
            float M = sM[0][q];
#pragma unroll
            for (int w = 1; w < 4; ++w) M = fmaxf(M, sM[w][q]);
            const float Ms = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float e = __builtin_amdgcn_exp2f(sM[w][q] - Ms);
                const float4 v = *reinterpret_cast<const float4*>(&sO[w][q][d]);
                L = fmaf(e, sL[w][q], L);
                O.x = fmaf(e, v.x, O.x);
                O.y = fmaf(e, v.y, O.y);
                O.z = fmaf(e, v.z, O.z);
                O.w = fmaf(e, v.w, O.w);
            }
            const int head = h * G + q0 + q;
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.0f / L;
                const size_t at = ((size_t)b * a.Hq + head) * D + d;
                if constexpr (KIND == A_F32)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                        make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                        make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
                if (a.lse && d == 0) a.lse[(size_t)b * a.Hq + head] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
            } else {
                const size_t pr = prow * a.Hq + head;
                *reinterpret_cast<float4*>(a.parts + pr * D + d) = O;
                if (d == 0)
                    *reinterpret_cast<float2*>(a.parts + a.p.rows * a.Hq * D + pr * 2) = make_float2(M, L);
            }
        }
    }
}

// Join of a sequence's parts: a workgroup per (sequence, query head), or per
// (listed sequence in several parts, query head).  Groups of D/4 lanes take the
// parts in turn, kBatch at a time with all their loads in flight (without a list
// the first batch's before the number of parts is known: they lie in the
// workspace whether written or not), each group with its own running maximum;
// the groups are joined through LDS in a fixed order.
template <int KIND, int D, bool LISTED>
__global__ __launch_bounds__(256) void beam_attn_join(AttnDecodeArgs a) {
    constexpr int LPR = D / 4, NG = 256 / LPR, kBatch = 4;
    __shared__ float sO[NG][D];
    __shared__ float sM[NG], sL[NG];
    const int head = blockIdx.x % a.Hq, grp = threadIdx.x / LPR, d = threadIdx.x % LPR * 4;
    int b = blockIdx.x / a.Hq, last = (int)a.p.S - 1;
    size_t row = (size_t)b * a.p.S;
    if constexpr (LISTED) {
        const int4 list = a.lists[b];
        if (list.x < 0) return;
        b = list.x;
        row = list.y;
        last = list.z - 1;
    }
    const float2* ml = reinterpret_cast<const float2*>(a.parts + a.p.rows * a.Hq * D);
    const size_t first = row * a.Hq + head, result = (size_t)b * a.Hq + head;
    float2 v[kBatch];
    float4 o[kBatch];
    auto load = [&](int s0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const size_t pr = first + (size_t)min(s0 + k * NG, last) * a.Hq;
            v[k] = ml[pr];
            o[k] = *reinterpret_cast<const float4*>(a.parts + pr * D + d);
        }
    };
    load(grp);
    const int n = LISTED ? last + 1 : span_of<false>(a, table_tokens(a), a.lens[b]).n;
    if (n <= 1) return;                           // its only part wrote the result
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = grp; s0 < n; s0 += kBatch * NG) {
        if (s0 != grp) load(s0);
        float top = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (s0 + k * NG < n) top = fmaxf(top, v[k].x);
        const float ts = top == -INFINITY ? 0.f : top;
        const float alpha = __builtin_amdgcn_exp2f(M - ts);
        M = top;
        L *= alpha;
        O.x *= alpha; O.y *= alpha; O.z *= alpha; O.w *= alpha;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (s0 + k * NG < n) {
                const float e = __builtin_amdgcn_exp2f(v[k].x - ts);
                L = fmaf(e, v[k].y, L);
                O.x = fmaf(e, o[k].x, O.x);
                O.y = fmaf(e, o[k].y, O.y);
                O.z = fmaf(e, o[k].z, O.z);
                O.w = fmaf(e, o[k].w, O.w);
            }
    }
    *reinterpret_cast<float4*>(&sO[grp][d]) = O;
    if (d == 0) {
        sM[grp] = M;
        sL[grp] = L;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t >= D) return;
    float top = sM[0];
#pragma unroll
    for (int k = 1; k < NG; ++k) top = fmaxf(top, sM[k]);
    const float ts = top == -INFINITY ? 0.f : top;
    float Lt = 0.f, Ot = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        const float e = __builtin_amdgcn_exp2f(sM[k] - ts);
        Lt = fmaf(e, sL[k], Lt);
        Ot = fmaf(e, sO[k][t], Ot);
    }
    const float res = Lt == 0.f ? 0.f : Ot / Lt;
    const size_t at = result * D + t;
    if constexpr (KIND == A_F32) static_cast<float*>(a.out)[at] = res;
    else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(res);
    if (a.lse && t == 0) a.lse[result] = Lt == 0.f ? -INFINITY : top * kLn2 + logf(Lt);
}

template <int KIND, int D, int QT>
static hipError_t launch_decode(const AttnDecodeArgs& a, hipStream_t st) {
    const int qgroups = (a.G + 16 * QT - 1) / (16 * QT);
    const size_t bh = (a.p.extra ? a.p.rows : (size_t)a.B) * a.Hkv;
    const unsigned grid = (unsigned)(qgroups == 1 ? bh : (bh + 7) / 8 * 8 * qgroups);
    const dim3 heads((unsigned)((size_t)a.p.joins * a.Hq));
    hipError_t err;
    if (a.p.extra) {
        err = launch(beam_attn_list, dim3(1), dim3(kListThreads), st, a);
        if (err == hipSuccess) err = launch(beam_attn_decode<KIND, D, QT, true>, dim3(grid), dim3(256), st, a, qgroups);
        return err == hipSuccess ? launch(beam_attn_join<KIND, D, true>, heads, dim3(256), st, a) : err;
    }
    err = launch(beam_attn_decode<KIND, D, QT, false>, dim3(grid, a.p.S), dim3(256), st, a, qgroups);
    if (err != hipSuccess || a.p.S == 1) return err;
    return launch(beam_attn_join<KIND, D, false>, heads, dim3(256), st, a);
}

// Above 16 queries per key-value head a wave takes 32 at once, so the cache
// is read half as often; at D = 256 their sums would not fit the registers.
template <int KIND>
static hipError_t launch_decode_d(const AttnDecodeArgs& a, hipStream_t st) {
    const bool wide = a.G > 16;
    if (a.D == 64) return wide ? launch_decode<KIND, 64, 2>(a, st) : launch_decode<KIND, 64, 1>(a, st);
    if (a.D == 128) return wide ? launch_decode<KIND, 128, 2>(a, st) : launch_decode<KIND, 128, 1>(a, st);
    return launch_decode<KIND, 256, 1>(a, st);
}

hipError_t launch_attn_decode(AttnDecodeArgs a, void* ws, hipStream_t st) {
    a.parts = static_cast<float*>(ws);
    if (a.p.extra) {
        a.items = static_cast<int4*>(ws);
        a.lists = a.items + a.p.rows;
        a.parts = reinterpret_cast<float*>(a.lists + a.p.joins);
    }
    if (a.c.kind == A_F32) return launch_decode_d<A_F32>(a, st);
    if (a.c.kind == A_BF16) return launch_decode_d<A_BF16>(a, st);
    return launch_decode_d<A_FP8>(a, st);
}

}  // namespace beam
