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
// The cache's length is split over workgroups (S parts per sequence) and over
// the four waves of a workgroup (32-token tiles in turn).  The waves' results
// are joined through LDS, the parts' through the workspace by a second
// kernel.
#include "common.h"
#include "kernels.h"

namespace beam {

constexpr int kTile = 32;            // tokens per wave step
constexpr int kStep = 4 * kTile;     // tokens per workgroup step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Parts of a sequence: about kWantWG workgroups in all, each of whole steps.
constexpr int kWantWG = 1024;
void attn_decode_split(int B, int Hkv, int max_len, int window, int* S, int* C) {
    // a window's tokens start inside a tile
    const int64_t span = window > 0 && window < max_len ? (int64_t)window + kTile - 1 : max_len;
    const int64_t heads = (int64_t)B * Hkv;
    const int64_t want = (kWantWG + heads - 1) / heads;
    int64_t c = (span + want - 1) / want;
    c = (c + kStep - 1) / kStep * kStep;
    if (c < kStep) c = kStep;
    int64_t s = (span + c - 1) / c;
    if (s < 1) s = 1;
    *S = (int)s;
    *C = (int)c;
}

size_t attn_decode_ws_bytes(int B, int Hq, int Hkv, int D, int max_len, int window) {
    int S, C;
    attn_decode_split(B, Hkv, max_len, window, &S, &C);
    return S > 1 ? (size_t)B * S * Hq * (D + 2) * sizeof(float) : 0;
}

// Tokens [t0, t1) of part s of a sequence.  Every part has at least C tokens
// and together they cover the sequence whatever its length.
struct Span {
    int start, t0, t1, n;   // first token seen; the part's range; parts that have tokens
};
BEAM_DEV Span span_of(const AttnDecodeArgs& a, int b, int s) {
    const int64_t cap = min((int64_t)a.max_pages << a.c.pshift, (int64_t)kMaxLen);
    const int len = (int)min((int64_t)max(a.lens[b], 0), cap);
    Span p;
    p.start = a.window > 0 ? max(0, len - a.window) : 0;
    const int base = p.start & ~(kTile - 1);
    const int all = len - base;
    const int64_t per = ((int64_t)all + a.S - 1) / a.S;
    const int64_t chunk = max((int64_t)a.C, (per + kStep - 1) & ~(int64_t)(kStep - 1));
    p.n = (int)((all + chunk - 1) / chunk);
    p.t0 = (int)min((int64_t)len, base + min(s, p.n) * chunk);
    p.t1 = (int)min((int64_t)len, p.t0 + chunk);
    return p;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// eight e4m3 codes to bf16 (exact)
BEAM_DEV void e4m3_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const f32x2 p = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), q = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    lo = pack_bf16x2(p.x, p.y);
    hi = pack_bf16x2(q.x, q.y);
}

// NW 32-bit words from global memory (16-, 8- or 4-byte pieces)
template <int NW> BEAM_DEV void ldw(const void* p, uint32_t (&w)[NW]) {
    if constexpr (NW % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i) {
            const uint4 v = static_cast<const uint4*>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (NW == 2) {
        const uint2 v = *static_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        static_assert(NW == 1, "");
        w[0] = *static_cast<const uint32_t*>(p);
    }
}

template <int KIND, int D>
__global__ __launch_bounds__(256) void beam_attn_decode(AttnDecodeArgs a, int qtiles) {
    constexpr int ES = KIND == A_F32 ? 4 : (KIND == A_BF16 ? 2 : 1);   // bytes per cache element
    constexpr int DL = D / 16;                    // value elements per lane and token
    constexpr int NQ = KIND == A_F32 ? D / 16 : D / 32;   // K fragments per token row
    constexpr int QW = 4;                         // words per query fragment
    __shared__ float sO[4][16][D + 4];
    __shared__ float sM[4][16], sL[4][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    int id = blockIdx.x;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int qt = id % qtiles;
    id /= qtiles;
    const int s = id % a.S, b = id / a.S;
    const int G = a.Hq / a.Hkv;
    const int P = 1 << a.c.pshift;
    const Span sp = span_of(a, b, s);
    if (s > 0 && s >= sp.n) return;               // no tokens; part 0 of an empty row goes on

    // query fragments: lane (r, g) holds column r (head h*G + 16 qt + r)
    const int qrow = qt * 16 + r;
    const size_t qoff = (size_t)b * a.qs + (size_t)(h * G + qrow) * D;
    uint32_t qf[NQ][QW];
#pragma unroll
    for (int c = 0; c < NQ; ++c) {
        if (qrow < G) {
            if constexpr (KIND == A_F32) ldw<4>(static_cast<const float*>(a.q) + qoff + 16 * c + 4 * g, qf[c]);
            else ldw<4>(static_cast<const uint16_t*>(a.q) + qoff + 32 * c + 8 * g, qf[c]);
        } else {
#pragma unroll
            for (int j = 0; j < QW; ++j) qf[c][j] = 0u;
        }
    }

    f32x4 o[DL];
#pragma unroll
    for (int t = 0; t < DL; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const float zs = a.scale * kLog2e;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    const uint8_t* kc = static_cast<const uint8_t*>(a.c.k);
    const uint8_t* vc = static_cast<const uint8_t*>(a.c.v);

    for (int tile = sp.t0 + wave * kTile; tile < sp.t1; tile += kStep) {
        // the two 16-token blocks' first cache rows; a block past the end or
        // on a bad page reads page 0 and is masked
        size_t row[2];
        bool ok[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tok = tile + 16 * u;
            int page = -1;
            if (tok < sp.t1) page = table[tok >> a.c.pshift];
            ok[u] = page >= 0 && page < a.c.n_pages;
            row[u] = (((size_t)(ok[u] ? page : 0) * a.Hkv + h) << a.c.pshift) + (tok & (P - 1));
        }
        f32x4 z[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            z[u] = f32x4{0.f, 0.f, 0.f, 0.f};
            const uint8_t* kr = kc + (row[u] + r) * (D * ES);
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                if constexpr (KIND == A_F32) {
                    uint32_t w[4];
                    ldw<4>(kr + (16 * c + 4 * g) * 4, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]), __uint_as_float(qf[c][e]),
                                                                    z[u], 0, 0, 0);
                } else {
                    uint4 w;
                    if constexpr (KIND == A_BF16) {
                        w = *reinterpret_cast<const uint4*>(kr + (32 * c + 8 * g) * 2);
                    } else {
                        uint32_t f[2];
                        ldw<2>(kr + 32 * c + 8 * g, f);
                        e4m3_to_bf16(f[0], w.x, w.y);
                        e4m3_to_bf16(f[1], w.z, w.w);
                    }
                    const uint4 qv = make_uint4(qf[c][0], qf[c][1], qf[c][2], qf[c][3]);
                    z[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                                   __builtin_bit_cast(bf16x8, qv), z[u], 0, 0, 0);
                }
            }
        }
        // scores in powers of two; lane: query r, tokens 16u + 4g + i
        float zz[2][4];
        bool live[2][4];
        float4 vs[2];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float4 ks = make_float4(1.f, 1.f, 1.f, 1.f);
            vs[u] = ks;
            if constexpr (KIND == A_FP8) {
                ks = *reinterpret_cast<const float4*>(a.c.ks + row[u] + 4 * g);
                vs[u] = *reinterpret_cast<const float4*>(a.c.vs + row[u] + 4 * g);
            }
            const float kss[4] = {ks.x, ks.y, ks.z, ks.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = tile + 16 * u + 4 * g + i;
                live[u][i] = ok[u] && tok >= sp.start && tok < sp.t1;
                zz[u][i] = live[u][i] ? z[u][i] * kss[i] * zs : -INFINITY;
                top = fmaxf(top, zz[u][i]);
            }
        }
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float mn = fmaxf(m, top);
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float alpha = __builtin_amdgcn_exp2f(m - ms);
        m = mn;
        float p[2][4];
        float ps = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[u][i] = __builtin_amdgcn_exp2f(zz[u][i] - ms);   // masked: exp2(-inf) = 0
                ps += p[u][i];
            }
        l = l * alpha + ps;
#pragma unroll
        for (int t = 0; t < DL; ++t) o[t] *= alpha;

        // values of this lane's tokens; a masked token's row may hold anything
        if constexpr (KIND == A_F32) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[DL];
                    ldw<DL>(vc + ((row[u] + 4 * g + i) * D + r * DL) * 4, w);
#pragma unroll
                    for (int t = 0; t < DL; ++t)
                        o[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(live[u][i] ? __uint_as_float(w[t]) : 0.f, p[u][i],
                                                                    o[t], 0, 0, 0);
                }
        } else {
            uint32_t v[8][DL / 2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* vr = vc + ((row[u] + 4 * g + i) * D + r * DL) * ES;
                    if constexpr (KIND == A_BF16) {
                        ldw<DL / 2>(vr, v[4 * u + i]);
                    } else {
                        uint32_t f[DL / 4];
                        ldw<DL / 4>(vr, f);
#pragma unroll
                        for (int j = 0; j < DL / 4; ++j) e4m3_to_bf16(f[j], v[4 * u + i][2 * j], v[4 * u + i][2 * j + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < DL / 2; ++j) v[4 * u + i][j] = live[u][i] ? v[4 * u + i][j] : 0u;
                    // the value scale joins the probability (one rounding to bf16)
                    if constexpr (KIND == A_FP8) {
                        const float vss[4] = {vs[u].x, vs[u].y, vs[u].z, vs[u].w};
                        p[u][i] *= live[u][i] ? vss[i] : 0.f;
                    }
                }
            const uint4 pw = make_uint4(pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                                        pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3]));
#pragma unroll
            for (int t = 0; t < DL; ++t) {
                const uint32_t sel = t % 2 ? 0x07060302u : 0x05040100u;
                uint4 w;
                w.x = __builtin_amdgcn_perm(v[1][t / 2], v[0][t / 2], sel);
                w.y = __builtin_amdgcn_perm(v[3][t / 2], v[2][t / 2], sel);
                w.z = __builtin_amdgcn_perm(v[5][t / 2], v[4][t / 2], sel);
                w.w = __builtin_amdgcn_perm(v[7][t / 2], v[6][t / 2], sel);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                               __builtin_bit_cast(bf16x8, pw), o[t], 0, 0, 0);
            }
        }
    }

    // join the four waves: o[t][i] of lane (r, g) is query r, d = (4g + i) * DL + t
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if (g == 0) {
        sM[wave][r] = m;
        sL[wave][r] = l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < DL; ++t) sO[wave][r][(4 * g + i) * DL + t] = o[t][i];
    __syncthreads();
    const int rows = min(16, G - qt * 16);
    for (int x = threadIdx.x; x < rows * (D / 4); x += 256) {
        const int q = x / (D / 4), d = x % (D / 4) * 4;
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
        const int head = h * G + qt * 16 + q;
        if (a.S == 1) {
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
            const size_t pr = ((size_t)b * a.S + s) * a.Hq + head;
            *reinterpret_cast<float4*>(a.parts + pr * D + d) = O;
            if (d == 0)
                *reinterpret_cast<float2*>(a.parts + (size_t)a.B * a.S * a.Hq * D + pr * 2) = make_float2(M, L);
        }
    }
}

// Join of a sequence's parts: one wave per (sequence, query head), D/64
// elements per lane, parts in order.
template <bool BF, int D>
__global__ __launch_bounds__(256) void beam_attn_join(AttnDecodeArgs a) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63;
    const int wid = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wid >= a.B * a.Hq) return;
    const int b = wid / a.Hq, head = wid - b * a.Hq;
    const int n = max(span_of(a, b, 0).n, 1);
    const float2* ml = reinterpret_cast<const float2*>(a.parts + (size_t)a.B * a.S * a.Hq * D);
    const size_t first = (size_t)b * a.S * a.Hq + head;
    float M = -INFINITY;
    for (int s = 0; s < n; ++s) M = fmaxf(M, ml[first + (size_t)s * a.Hq].x);
    const float Ms = M == -INFINITY ? 0.f : M;
    float L = 0.f, O[N];
#pragma unroll
    for (int j = 0; j < N; ++j) O[j] = 0.f;
    for (int s = 0; s < n; ++s) {
        const size_t pr = first + (size_t)s * a.Hq;
        const float2 v = ml[pr];
        const float e = __builtin_amdgcn_exp2f(v.x - Ms);
        L = fmaf(e, v.y, L);
#pragma unroll
        for (int j = 0; j < N; ++j) O[j] = fmaf(e, a.parts[pr * D + j * 64 + lane], O[j]);
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const size_t at = (size_t)wid * D + j * 64 + lane;
        if constexpr (BF) static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(O[j] * inv);
        else static_cast<float*>(a.out)[at] = O[j] * inv;
    }
    if (a.lse && lane == 0) a.lse[wid] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

template <int KIND, int D>
static hipError_t launch_decode(const AttnDecodeArgs& a, hipStream_t st) {
    const int qtiles = (a.Hq / a.Hkv + 15) / 16;
    const unsigned grid = (unsigned)((size_t)a.B * a.S * qtiles * a.Hkv);
    hipLaunchKernelGGL((beam_attn_decode<KIND, D>), dim3(grid), dim3(256), 0, st, a, qtiles);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.S == 1) return err;
    const dim3 jgrid((a.B * a.Hq + 3) / 4);
    hipLaunchKernelGGL((beam_attn_join<KIND != A_F32, D>), jgrid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int KIND>
static hipError_t launch_decode_d(const AttnDecodeArgs& a, hipStream_t st) {
    if (a.D == 64) return launch_decode<KIND, 64>(a, st);
    if (a.D == 128) return launch_decode<KIND, 128>(a, st);
    return launch_decode<KIND, 256>(a, st);
}

hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t st) {
    if (a.c.kind == A_F32) return launch_decode_d<A_F32>(a, st);
    if (a.c.kind == A_BF16) return launch_decode_d<A_BF16>(a, st);
    return launch_decode_d<A_FP8>(a, st);
}

}  // namespace beam
