// What goes into the attention: per-head RMSNorm of queries and keys, the
// position rotation, the queries' position factor, and the paged key-value
// cache (written in bf16, fp32, e4m3 or 4 bits, and read back).
// (TokenSpeed x Reflection Beam blog, "Architecture", and vLLM Beam summary,
//  kernel list: QK norm + rotation or position factor in one kernel with the
//  cache write.)
//
// A head row is spread over D/8 lanes of 8 consecutive elements, so a wave
// holds 512/D heads, a row's sums take log2(D/8) lane exchanges and every
// access is 16 bytes of bf16 per lane.
#include "attn_common.h"

namespace beam {

// ---------------------------------------------------------------- 8 elements

template <bool BF> struct Raw8;
template <> struct Raw8<true> { uint4 v; };
template <> struct Raw8<false> { float4 a, b; };

template <bool BF> BEAM_DEV Raw8<BF> ld8(const void* p, size_t i) {
    Raw8<BF> r;
    if constexpr (BF) {
        r.v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        r.a = f[0];
        r.b = f[1];
    }
    return r;
}
BEAM_DEV void wid8(const Raw8<true>& r, float (&x)[8]) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}
BEAM_DEV void wid8(const Raw8<false>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
template <bool BF> BEAM_DEV void st8(void* p, size_t i, const float (&x)[8]) {
    if constexpr (BF) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
    } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// value of the lane that the DPP control CTRL gives inside rows of 16 lanes
template <int CTRL> BEAM_DEV float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140, kRor8 = 0x128;

// Combines over the LPH lanes that hold one head row, every lane getting the
// result: pairs, quads, then the mirror image of 8 and of 16 lanes (whose
// other half already agrees among itself) by DPP, and 16 lanes further by the
// row swap.
template <int LPH, typename F> BEAM_DEV float head_reduce(float v, F f) {
    v = f(v, dpp<kXor1>(v));
    v = f(v, dpp<kXor2>(v));
    v = f(v, dpp<kHalfMirror>(v));
    if constexpr (LPH >= 16) v = f(v, dpp<kMirror>(v));
    if constexpr (LPH >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
    }
    return v;
}
template <int LPH> BEAM_DEV float head_sum(float v) {
    return head_reduce<LPH>(v, [](float a, float b) { return a + b; });
}
template <int LPH> BEAM_DEV float head_max(float v) {
    return head_reduce<LPH>(v, [](float a, float b) { return fmaxf(a, b); });
}

// The 8 quotients x / s, correctly rounded.  They share s, so its reciprocal
// is formed once, by a Newton step, and each quotient takes a product and a
// correction by its exact remainder (Markstein 1990).  That leaves a quotient
// wrong only if it lies within 3/2 units (of 2^-24 of the divisor's) of a
// midpoint between two floats; of those cases, which were all gone through, none
// comes out wrong with a correctly rounded reciprocal, and with the float on
// its other side only four, whose divisors' significands are the last before 2.
// Those, and an s with which a step could leave the range of normal numbers,
// take __fdiv_rn.  The remainder is formed negative and taken times -y: so the
// signs of -0 and of a NaN stay.
BEAM_DEV void divide8(float (&x)[8], float s) {
    if (__any(!(s > 1e-25f && s < 1e25f) || (__float_as_uint(s) & 0x7FFFF8u) == 0x7FFFF8u)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], s);
        return;
    }
    const float y0 = __builtin_amdgcn_rcpf(s);
    const float y = fmaf(fmaf(-s, y0, 1.0f), y0, y0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float q = x[j] * y;
        x[j] = fmaf(fmaf(q, s, -x[j]), -y, q);
    }
}

// 1 / sqrt(s), half a unit in the last place off but for 2^-20 of one: the
// hardware's estimate and a Newton step whose residual 1 - s y^2 is formed from
// the exact product s y = h + l.  (A rounded root and a rounded quotient of it
// are up to 1.3 off: an fp32 norm was 5.8e-8 from the exact one, now 5.2e-8.)
BEAM_DEV float inv_sqrt(float s) {
    if (!(s > 1e-30f && s < 1e30f)) return 1.0f / sqrtf(s);   // 0, infinite and NaN too
    const float y = __builtin_amdgcn_rsqf(s);
    const float h = s * y, l = fmaf(s, y, -h);
    const float e = fmaf(-l, y, fmaf(-h, y, 1.0f));
    return fmaf(0.5f * e, y, y);
}

// Stores a head row's 8 elements of this lane at row `row` of one cache
// side.  e4m3: the scale and codes that quantize_row_e4m3_wave gives a row.  4
// bits: per block of 32 elements, four lanes', the E8M0 byte of floor(log2 amax)
// - 2 (at least 0; the exponent field of amax less 2) and E2M1 codes: what
// beam_quantize_mx_rows gives a finite block.  A NaN counts as 0 in amax and is
// stored as +-6 times the scale, an infinite element likewise with the largest
// scale there is, 2^126: it reads back as infinite.
template <int CK, int D>
BEAM_DEV void store_cache(void* side, void* scales, size_t row, int e0, float (&x)[8], bool live) {
    if constexpr (CK == A_FP4) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
        amax = fmaxf(amax, dpp<kXor1>(amax));   // every lane takes part
        amax = fmaxf(amax, dpp<kXor2>(amax));
        const int byte = max((int)(__float_as_uint(amax) >> 23) - 2, 0);
        const float s = e8m0((uint32_t)byte);
        if (!live) return;
        uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(side) + row * (D / 2) + e0 / 2) = c;
        if (e0 % 32 == 0) static_cast<uint8_t*>(scales)[row * (D / 32) + e0 / 32] = (uint8_t)byte;
    } else if constexpr (CK == A_FP8) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
        amax = head_max<D / 8>(amax);   // every lane takes part
        const float top = __fdiv_rn(amax, 448.0f);
        const float s = top > 0.f ? top : 1.0f;   // 0 too where amax / 448 is less than half the least float
        divide8(x, s);
        if (!live) return;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(side) + row * D + e0) =
            make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
        if (e0 == 0) static_cast<float*>(scales)[row] = s;
    } else {
        if (live) st8<CK == A_BF16>(side, row * D + e0, x);
    }
}

// ---------------------------------------------------------------------------
// Units of a token: its Hq query heads, Hkv key heads and (into the cache)
// Hkv value heads, in that order.  A wave takes `gpw` consecutive groups of
// 512/D units of one token; the rotation's cosines and sines depend on the
// lane's place in the head only, so they are formed once per wave, one or two
// frequencies per lane, and handed round.
//   For a row x: y = R(x * gamma) * f, with f = 1/sqrt(mean(x^2) + eps) times
// the position factor: the rotation R is linear, so both factors wait until
// after it.  Bound by HBM where there are many tokens (16384 of 48 + 8 + 8 heads
// of 128, bf16 into e4m3: 97 us, 5.2 TB/s; values and keys alone: 22.7 us, 4.5
// TB/s; a copy reaches 4.7), by latency where there are few (64: 3.8 us).  Into 4
// bits: 92 us with norm and rotation (e4m3 96, bf16 100); values and keys alone, and
// back, 40 us in two launches.
// ---------------------------------------------------------------------------
template <bool BF, int CK, int D>
__global__ __launch_bounds__(256) void beam_attn_prep(AttnPrepArgs a, int units, int wpt, int gpw) {
    constexpr int LPH = D / 8, HPW = kWave / LPH;
    const int lane = threadIdx.x & 63;
    const int wid = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = wid / wpt;
    if (t >= a.T) return;   // whole wave
    const int g0 = (wid - t * wpt) * gpw;
    const int gend = min(g0 + gpw, (units + HPW - 1) / HPW);
    const int li = lane % LPH, e0 = li * 8;

    // this lane's place in each matrix's row of the token
    const size_t esz = BF ? 2 : 4;
    const char* qrow = static_cast<const char*>(a.q) + ((size_t)t * a.qs + e0) * esz;
    const char* krow = static_cast<const char*>(a.k) + ((size_t)t * a.ks + e0) * esz;
    const char* vrow = static_cast<const char*>(a.v) + ((size_t)t * a.vs + e0) * esz;
    auto load = [&](int gi) {   // lanes past the last unit load it again
        const int u = min(gi * HPW + lane / LPH, units - 1);
        const char* p = qrow + (size_t)u * (D * esz);
        if ((gi + 1) * HPW > a.Hq) {
            const int k = u - a.Hq, v = k - a.Hkv;
            p = k < 0 ? p : (v < 0 ? krow + (size_t)k * (D * esz) : vrow + (size_t)v * (D * esz));
        }
        return ld8<BF>(p, 0);
    };
    Raw8<BF> next = load(g0);   // a group's loads are in flight while the group before it is worked on

    // The angles' cosines and sines for this lane's elements: half-split,
    // element e0 + j of the rotated dims has frequency (e0 + j) mod R/2, and
    // the sine enters the lower half with a minus; interleaved, the pair
    // (e0 + 2j, e0 + 2j + 1) has frequency e0/2 + j.
    float cs[8], sn[8];
    const int half = a.R / 2;
    const bool turns = e0 < a.R;
    if (a.R > 0) {
        const double p = (double)a.pos[t];
        float c[2], s[2];
        auto angle = [&](int k) {
            // whole turns drop out in fp64, so far positions keep their angle;
            // what fp32 then leaves of it enters to first order
            double rev = p * ((double)a.inv_freq[min(lane + 64 * k, half - 1)] * 0.15915494309189533577);
            rev -= rint(rev);
            const float turn = (float)(2.0 * rev);
            const float rest = (float)(2.0 * rev - (double)turn) * 3.14159265f;
            float s0, c0;
            sincospif(turn, &s0, &c0);
            s[k] = fmaf(c0, rest, s0);
            c[k] = fmaf(-s0, rest, c0);
        };
        angle(0);
        if (D > 128 && half > 64) angle(1);
        const int f0 = a.inter ? e0 / 2 : (e0 < half ? e0 : e0 - half);
        const float sg = !a.inter && e0 < half ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int f = f0 + j;
            cs[j] = __shfl(c[0], f & 63, kWave);
            sn[j] = __shfl(s[0], f & 63, kWave);
            if (D > 128 && half > 64) {
                const float c1 = __shfl(c[1], f & 63, kWave), s1 = __shfl(s[1], f & 63, kWave);
                cs[j] = f >= 64 ? c1 : cs[j];
                sn[j] = f >= 64 ? s1 : sn[j];
            }
            sn[j] *= sg;
        }
    }
    float qf = 1.f;
    if (a.ssmax_len > 0.f) qf = powf(1.f + fmaxf((float)a.pos[t], 0.f) / a.ssmax_len, a.ssmax_exp);
    int slot = -1;
    if (CK >= 0) {
        slot = a.slots[t];
        if ((int64_t)slot >= ((int64_t)a.c.n_pages << a.c.pshift)) slot = -1;
    }
    float g[8];
    if (a.gq) wid8(ld8<BF>(a.gq, e0), g);
    bool g_is_q = true;

    for (int gi = g0; gi < gend; ++gi) {
        const int u = gi * HPW + lane / LPH;
        const bool only_q = (gi + 1) * HPW <= a.Hq;   // the same for the whole wave
        const bool is_q = only_q || u < a.Hq;
        const bool is_v = !only_q && u >= a.Hq + a.Hkv;
        float x[8];
        wid8(next, x);
        if (gi + 1 < gend) next = load(gi + 1);
        float f = 1.f;
        if (a.gq) {
            if (!only_q && g_is_q) {   // units only go on from queries to keys to values
                float gk[8];
                wid8(ld8<BF>(a.gk, e0), gk);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = is_q ? g[j] : gk[j];
                g_is_q = gi * HPW < a.Hq;   // lanes of this group that are queries change at the next
            }
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            ss = head_sum<LPH>(ss);
            if (!is_v) {
                f = inv_sqrt(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= g[j];
            }
        }
        if (a.R > 0) {
            if (a.inter) {
                if (!is_v && turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float u0 = x[2 * j], w0 = x[2 * j + 1];
                        x[2 * j] = u0 * cs[j] - w0 * sn[j];
                        x[2 * j + 1] = w0 * cs[j] + u0 * sn[j];
                    }
                }
            } else {
                const int d = a.R / 16;   // lanes between the two elements of a pair
                float o[8];
                if (d == 8) {             // the other half of a row of 16 lanes
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = dpp<kRor8>(x[j]);
                } else {
                    const int from = turns ? (e0 < half ? lane + d : lane - d) : lane;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __shfl(x[j], from, kWave);
                }
                if (!is_v && turns) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = fmaf(o[j], sn[j], x[j] * cs[j]);
                }
            }
        }
        if (is_q) f *= qf;
        if (!is_v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f;
        }
        if (is_q) st8<BF>(a.q_out, ((size_t)t * a.Hq + u) * D + e0, x);
        if (only_q) continue;
        const bool kv = !is_q && u < units;   // lanes past the last unit store nothing
        const int h = is_v ? u - a.Hq - a.Hkv : u - a.Hq;
        if constexpr (CK < 0) {
            if (kv) st8<BF>(a.k_out, ((size_t)t * a.Hkv + h) * D + e0, x);
        } else {
            const size_t page = slot >= 0 ? (size_t)(slot >> a.c.pshift) : 0;
            const size_t row = ((page * a.Hkv + h) << a.c.pshift) + (slot & ((1 << a.c.pshift) - 1));
            store_cache<CK, D>(is_v ? a.c.v : a.c.k, is_v ? a.c.vs : a.c.ks, row, e0, x, kv && slot >= 0);
        }
    }
}

constexpr int kPrepWaves = 32768;

template <bool BF, int CK, int D>
static hipError_t launch_prep(const AttnPrepArgs& a, hipStream_t st) {
    constexpr int HPW = 512 / D;
    const int units = a.Hq + a.Hkv * (CK < 0 ? 1 : 2);
    const int groups = (units + HPW - 1) / HPW;
    // groups per wave: one while that leaves the chip with few waves, more
    // once the waves suffice, which forms a token's cosines fewer times (16384
    // tokens of 16 groups into an 8-bit cache: 124 us at 131072 waves, 106 at
    // 65536, 100 at 32768, 108 at 8192; no other size was swept)
    const int gpw = (int)min((int64_t)groups, max((int64_t)1, (int64_t)a.T * groups / kPrepWaves));
    const int wpt = (groups + gpw - 1) / gpw;
    const unsigned grid = (unsigned)(((size_t)a.T * wpt + 3) / 4);
    return launch(beam_attn_prep<BF, CK, D>, dim3(grid), dim3(256), st, a, units, wpt, gpw);
}

template <bool BF, int CK>
static hipError_t launch_prep_d(const AttnPrepArgs& a, hipStream_t st) {
    if (a.D == 64) return launch_prep<BF, CK, 64>(a, st);
    if (a.D == 128) return launch_prep<BF, CK, 128>(a, st);
    return launch_prep<BF, CK, 256>(a, st);
}

template <bool BF>
static hipError_t launch_prep_c(const AttnPrepArgs& a, hipStream_t st) {
    if (a.k_out) return launch_prep_d<BF, -1>(a, st);
    if (a.c.kind == A_F32) return launch_prep_d<BF, A_F32>(a, st);
    if (a.c.kind == A_BF16) return launch_prep_d<BF, A_BF16>(a, st);
    if (a.c.kind == A_FP4) return launch_prep_d<BF, A_FP4>(a, st);
    return launch_prep_d<BF, A_FP8>(a, st);
}

hipError_t launch_attn_prep(const AttnPrepArgs& a, hipStream_t st) {
    return a.bf16 ? launch_prep_c<true>(a, st) : launch_prep_c<false>(a, st);
}

// ---------------------------------------------------------------------------
// Cache rows back to dense rows.  A workgroup takes `rows` consecutive
// output rows: each lane finds one row's place in the cache, then groups of
// D/8 lanes copy one head row of one side at a time, kReadBatch of them with
// all their loads in flight.  Bound by HBM (91500 rows of 8 heads of 128, e4m3
// to bf16: 110 us, 5.2 TB/s; 4 bits to bf16, 474 MB: 103 us, 4.6 TB/s, most of it
// the rows written; one row per workgroup: 137 us; 4 rows and loads
// at a time: 119 us; one head of 128 instead of 8: 17.6 us with the 64 rows it
// gets, 50 with 8).
// ---------------------------------------------------------------------------
template <int CK> struct RawC8;                       // 8 cache elements as stored
template <> struct RawC8<A_BF16> { Raw8<true> v; };
template <> struct RawC8<A_F32> { Raw8<false> v; };
template <> struct RawC8<A_FP8> { uint2 v; float s; };
template <> struct RawC8<A_FP4> { uint32_t v; uint32_t s; };
template <int CK> BEAM_DEV RawC8<CK> ld_cache8(const void* side, const void* scales, size_t row, int D, int e0) {
    RawC8<CK> r;
    if constexpr (CK == A_FP4) {
        r.v = __builtin_nontemporal_load(
            reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(side) + row * (D / 2) + e0 / 2));   // read once
        r.s = static_cast<const uint8_t*>(scales)[row * (D / 32) + e0 / 32];
    } else if constexpr (CK == A_FP8) {
        typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
        const u32x2v w = __builtin_nontemporal_load(
            reinterpret_cast<const u32x2v*>(static_cast<const uint8_t*>(side) + row * D + e0));   // read once
        r.v = make_uint2(w.x, w.y);
        r.s = static_cast<const float*>(scales)[row];
    } else {
        r.v = ld8<CK == A_BF16>(side, row * D + e0);
    }
    return r;
}
template <int CK> BEAM_DEV void wid_cache8(const RawC8<CK>& r, float (&x)[8]) {
    if constexpr (CK == A_FP4) {
        const float s = e8m0(r.s);   // exact in bf16, so in fp32 too
        const uint32_t w[4] = {e2m1_pair<0>(r.v, s), e2m1_pair<1>(r.v, s), e2m1_pair<2>(r.v, s), e2m1_pair<3>(r.v, s)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else if constexpr (CK == A_FP8) {
        typedef float f32x2v __attribute__((ext_vector_type(2)));
        const uint32_t w[2] = {r.v.x, r.v.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x2v lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
            const f32x2v hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
            x[4 * j] = lo.x * r.s;
            x[4 * j + 1] = lo.y * r.s;
            x[4 * j + 2] = hi.x * r.s;
            x[4 * j + 3] = hi.y * r.s;
        }
    } else {
        wid8(r.v, x);
    }
}

constexpr int kReadBatch = 8;

template <bool BF, int CK, int D>
__global__ __launch_bounds__(256) void beam_kv_read(KvReadArgs a, int rows) {
    constexpr int LPH = D / 8, HPB = 256 / LPH;
    const int lane = threadIdx.x & 63;
    const int row0 = blockIdx.x * rows;
    const int last = a.offsets[a.B];   // rows at and behind it stay
    if (row0 >= last) return;
    // lane i: cache row (of head 0) and page of output row row0 + i
    const int mine = row0 + min(lane, rows - 1);
    int lo = 0, hi = a.B;              // offsets[lo] <= mine < offsets[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.offsets[mid] <= mine) lo = mid;
        else hi = mid;
    }
    const int64_t tok = (int64_t)mine - a.offsets[lo] + (a.first ? a.first[lo] : 0);
    const int64_t pi = tok >> a.c.pshift;
    int page = -1;
    if (tok >= 0 && pi < a.max_pages) page = a.table[(size_t)lo * a.max_pages + pi];
    if (page >= a.c.n_pages) page = -1;
    const int off = (int)(tok & ((1 << a.c.pshift) - 1));

    const int e0 = (threadIdx.x % LPH) * 8;
    const int per_row = 2 * a.Hkv, n = min(rows, min(a.N, last) - row0) * per_row;
    for (int base = 0; base < n; base += kReadBatch * HPB) {
        RawC8<CK> v[kReadBatch];
        int row[kReadBatch], h[kReadBatch];
        bool is_v[kReadBatch], ok[kReadBatch];
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
            const int i = min(base + k * HPB + (int)threadIdx.x / LPH, n - 1);
            row[k] = i / per_row;
            h[k] = i - row[k] * per_row;
            is_v[k] = h[k] >= a.Hkv;
            if (is_v[k]) h[k] -= a.Hkv;
            const int pg = __shfl(page, row[k], kWave), at = __shfl(off, row[k], kWave);
            ok[k] = pg >= 0;
            const size_t from = (((size_t)(ok[k] ? pg : 0) * a.Hkv + h[k]) << a.c.pshift) + at;
            v[k] = ld_cache8<CK>(is_v[k] ? a.c.v : a.c.k, is_v[k] ? a.c.vs : a.c.ks, from, D, e0);
        }
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
            if (base + k * HPB + (int)threadIdx.x / LPH >= n) continue;
            float x[8];
            wid_cache8<CK>(v[k], x);
            if (!ok[k]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.f;
            }
            st8<BF>(is_v[k] ? a.v_out : a.k_out, ((size_t)(row0 + row[k]) * a.Hkv + h[k]) * D + e0, x);
        }
    }
}

// Rows of a workgroup: as many as give each thread kReadBatch loads (8 with 8
// heads of 128; at most the 64 that a wave's lanes look up), fewer where that
// leaves CUs without a workgroup, more where a launch could not hold the
// workgroups (it holds fewer than 2^32 threads).
constexpr int kReadWG = 512, kMostReadWG = 1 << 23;
int kv_read_rows(int N, int Hkv, int D) {
    int rows = 256 * kReadBatch / (2 * Hkv * (D / 8));
    rows = rows < 1 ? 1 : (rows > 64 ? 64 : rows);
    while (rows > 8 && N / rows < kReadWG) rows /= 2;
    const int least = (int)(((int64_t)N + kMostReadWG - 1) / kMostReadWG);   // 8 for the most rows of a call
    return rows < least ? least : rows;
}

template <bool BF, int CK>
static hipError_t launch_read_d(const KvReadArgs& a, hipStream_t st) {
    const int rows = kv_read_rows(a.N, a.Hkv, a.D);
    const dim3 grid((unsigned)(((size_t)a.N + rows - 1) / rows)), block(256);
    if (a.D == 64) return launch(beam_kv_read<BF, CK, 64>, grid, block, st, a, rows);
    if (a.D == 128) return launch(beam_kv_read<BF, CK, 128>, grid, block, st, a, rows);
    return launch(beam_kv_read<BF, CK, 256>, grid, block, st, a, rows);
}

template <bool BF>
static hipError_t launch_read_c(const KvReadArgs& a, hipStream_t st) {
    if (a.c.kind == A_F32) return launch_read_d<BF, A_F32>(a, st);
    if (a.c.kind == A_BF16) return launch_read_d<BF, A_BF16>(a, st);
    if (a.c.kind == A_FP4) return launch_read_d<BF, A_FP4>(a, st);
    return launch_read_d<BF, A_FP8>(a, st);
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t st) {
    return a.bf16 ? launch_read_c<true>(a, st) : launch_read_c<false>(a, st);
}

}  // namespace beam
