// C ABI entry points of the attention sublayer: argument validation,
// workspace carving and launches.  Every check runs on the host before
// anything is enqueued.
#include "beam_moe.h"

#include <math.h>

#include "kernels.h"

namespace {

constexpr int64_t kMaxT = 1 << 22;          // tokens or sequences per call
constexpr int64_t kMaxParts = 1 << 23;      // query heads times parts per decode call: a launch of 256-thread
                                            // workgroups holds fewer than 2^32 threads
constexpr int64_t kMaxGroups = 1 << 24;     // such workgroups

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

beam_status check_attn_cfg(const beam_moe_attn_cfg* c) {
    if (!c) return BEAM_ERR_INVALID_ARG;
    if (c->n_heads <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->rope_dim < 0 || c->window < 0 ||
        c->page_size <= 0)
        return BEAM_ERR_INVALID_ARG;
    if (c->rope_interleaved != 0 && c->rope_interleaved != 1) return BEAM_ERR_INVALID_ARG;
    if (!(c->ssmax_len >= 0.f) || !isfinite(c->ssmax_len) || !isfinite(c->ssmax_exp) ||
        !(c->softmax_scale > 0.f) || !isfinite(c->softmax_scale) || !(c->rms_eps >= 0.f) ||
        !isfinite(c->rms_eps))
        return BEAM_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BEAM_ERR_UNSUPPORTED;
    if (c->n_heads > 256 || c->n_heads % c->n_kv_heads != 0 || c->n_heads / c->n_kv_heads > 64)
        return BEAM_ERR_UNSUPPORTED;
    if (c->rope_dim > c->head_dim) return BEAM_ERR_INVALID_ARG;
    if (c->rope_dim % 16 != 0) return BEAM_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
        return BEAM_ERR_UNSUPPORTED;
    return BEAM_OK;
}

beam_status check_cache(const beam_moe_attn_cfg* c, const beam_moe_kv_cache* k, beam::KvCache& out) {
    if (!k || !k->k || !k->v || k->n_pages <= 0) return BEAM_ERR_INVALID_ARG;
    if (k->dtype != BEAM_F32 && k->dtype != BEAM_BF16 && k->dtype != BEAM_FP8_E4M3 && k->dtype != BEAM_MXFP4)
        return BEAM_ERR_INVALID_ARG;
    if (!aligned16(k->k) || !aligned16(k->v)) return BEAM_ERR_INVALID_ARG;
    if ((k->dtype == BEAM_FP8_E4M3 || k->dtype == BEAM_MXFP4) &&
        (!k->k_scale || !k->v_scale || !aligned16(k->k_scale) || !aligned16(k->v_scale)))
        return BEAM_ERR_INVALID_ARG;
    if ((int64_t)k->n_pages * c->page_size > 0x7FFFFFFF) return BEAM_ERR_UNSUPPORTED;
    int sh = 0;
    while ((1 << sh) < c->page_size) ++sh;
    out.k = k->k;
    out.v = k->v;
    out.ks = k->k_scale;
    out.vs = k->v_scale;
    out.n_pages = k->n_pages;
    out.pshift = sh;
    out.kind = k->dtype == BEAM_F32    ? beam::A_F32
               : k->dtype == BEAM_BF16 ? beam::A_BF16
               : k->dtype == BEAM_MXFP4 ? beam::A_FP4
                                        : beam::A_FP8;
    return BEAM_OK;
}

bool sinks_ok(int32_t n) { return n >= 0 && n <= beam::kMaxLen; }

bool act_dtype(beam_dtype d) { return d == BEAM_F32 || d == BEAM_BF16; }

// a strided [T, heads, D] input: present, 16-byte aligned rows that hold its heads
bool rows_ok(const void* p, int64_t stride, int64_t width) {
    return p && aligned16(p) && stride >= width && stride % 8 == 0 && stride <= (int64_t)1 << 31;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

size_t span_bytes(int64_t T, int64_t stride, int64_t width, size_t es) {
    return (size_t)((T - 1) * stride + width) * es;
}

// The parts of the norm/rotation calls that the dense and the cached form share.
beam_status prep_common(const beam_moe_attn_cfg* c, int32_t T, const void* q, int64_t qs, const void* k, int64_t ks,
                        beam_dtype dtype, const void* gq, const void* gk, const int32_t* positions,
                        const float* inv_freq, void* q_out, beam::AttnPrepArgs& a) {
    const int64_t D = c->head_dim;
    if (!rows_ok(q, qs, c->n_heads * D) || !rows_ok(k, ks, c->n_kv_heads * D)) return BEAM_ERR_INVALID_ARG;
    if ((gq == nullptr) != (gk == nullptr) || !aligned16(gq) || !aligned16(gk)) return BEAM_ERR_INVALID_ARG;
    if (!positions || !aligned4(positions) || (c->rope_dim > 0 && !inv_freq) || !aligned4(inv_freq))
        return BEAM_ERR_INVALID_ARG;
    if (!q_out || !aligned16(q_out)) return BEAM_ERR_INVALID_ARG;
    const size_t es = dtype == BEAM_BF16 ? 2 : 4;
    const size_t qo = (size_t)T * c->n_heads * D * es;
    const bool q_self = q_out == q && qs == c->n_heads * D;
    if (!q_self && overlap(q_out, qo, q, span_bytes(T, qs, c->n_heads * D, es))) return BEAM_ERR_INVALID_ARG;
    if (overlap(q_out, qo, k, span_bytes(T, ks, c->n_kv_heads * D, es))) return BEAM_ERR_INVALID_ARG;
    a.T = T;
    a.Hq = c->n_heads;
    a.Hkv = c->n_kv_heads;
    a.D = c->head_dim;
    a.R = c->rope_dim;
    a.inter = c->rope_interleaved != 0;
    a.bf16 = dtype == BEAM_BF16;
    a.ssmax_len = c->ssmax_len;
    a.ssmax_exp = c->ssmax_exp;
    a.eps = c->rms_eps;
    a.q = q;
    a.k = k;
    a.qs = (size_t)qs;
    a.ks = (size_t)ks;
    a.gq = gq;
    a.gk = gk;
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    return BEAM_OK;
}

beam_status ran(hipError_t e) { return e == hipSuccess ? BEAM_OK : BEAM_ERR_HIP; }

}  // namespace

extern "C" {

beam_status beam_moe_qk_norm_rope(const beam_moe_attn_cfg* cfg, int32_t T, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, beam_dtype dtype, const void* gamma_q,
                                  const void* gamma_k, const int32_t* positions, const float* inv_freq, void* q_out,
                                  void* k_out, void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (T < 0 || T > kMaxT || !act_dtype(dtype)) return BEAM_ERR_INVALID_ARG;
    if (T == 0) return BEAM_OK;
    beam::AttnPrepArgs a{};
    st = prep_common(cfg, T, q, q_stride, k, k_stride, dtype, gamma_q, gamma_k, positions, inv_freq, q_out, a);
    if (st != BEAM_OK) return st;
    if (!k_out || !aligned16(k_out)) return BEAM_ERR_INVALID_ARG;
    const size_t es = dtype == BEAM_BF16 ? 2 : 4;
    const int64_t kw = (int64_t)cfg->n_kv_heads * cfg->head_dim, qw = (int64_t)cfg->n_heads * cfg->head_dim;
    const size_t ko = (size_t)T * kw * es;
    const bool k_self = k_out == k && k_stride == kw;
    if (!k_self && overlap(k_out, ko, k, span_bytes(T, k_stride, kw, es))) return BEAM_ERR_INVALID_ARG;
    if (overlap(k_out, ko, q, span_bytes(T, q_stride, qw, es)) || overlap(k_out, ko, q_out, (size_t)T * qw * es))
        return BEAM_ERR_INVALID_ARG;
    a.k_out = k_out;
    return ran(beam::launch_attn_prep(a, static_cast<hipStream_t>(stream)));
}

beam_status beam_moe_qk_norm_rope_cache(const beam_moe_attn_cfg* cfg, int32_t T, const void* q, int64_t q_stride,
                                        const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                        beam_dtype dtype, const void* gamma_q, const void* gamma_k,
                                        const int32_t* positions, const float* inv_freq, const int32_t* slots,
                                        void* q_out, const beam_moe_kv_cache* cache, void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (T < 0 || T > kMaxT || !act_dtype(dtype)) return BEAM_ERR_INVALID_ARG;
    if (T == 0) return BEAM_OK;
    beam::AttnPrepArgs a{};
    st = prep_common(cfg, T, q, q_stride, k, k_stride, dtype, gamma_q, gamma_k, positions, inv_freq, q_out, a);
    if (st != BEAM_OK) return st;
    const int64_t kw = (int64_t)cfg->n_kv_heads * cfg->head_dim, qw = (int64_t)cfg->n_heads * cfg->head_dim;
    const size_t es = dtype == BEAM_BF16 ? 2 : 4;
    if (!rows_ok(v, v_stride, kw) || !slots || !aligned4(slots)) return BEAM_ERR_INVALID_ARG;
    if (overlap(q_out, (size_t)T * qw * es, v, span_bytes(T, v_stride, kw, es))) return BEAM_ERR_INVALID_ARG;
    st = check_cache(cfg, cache, a.c);
    if (st != BEAM_OK) return st;
    a.v = v;
    a.vs = (size_t)v_stride;
    a.slots = slots;
    return ran(beam::launch_attn_prep(a, static_cast<hipStream_t>(stream)));
}

beam_status beam_moe_kv_write(const beam_moe_attn_cfg* cfg, int32_t T, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, beam_dtype dtype, const int32_t* slots,
                              const beam_moe_kv_cache* cache, void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (T < 0 || T > kMaxT || !act_dtype(dtype)) return BEAM_ERR_INVALID_ARG;
    if (T == 0) return BEAM_OK;
    const int64_t kw = (int64_t)cfg->n_kv_heads * cfg->head_dim;
    if (!rows_ok(k, k_stride, kw) || !rows_ok(v, v_stride, kw) || !slots || !aligned4(slots))
        return BEAM_ERR_INVALID_ARG;
    beam::AttnPrepArgs a{};
    st = check_cache(cfg, cache, a.c);
    if (st != BEAM_OK) return st;
    a.T = T;
    a.Hq = 0;
    a.Hkv = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.bf16 = dtype == BEAM_BF16;
    a.k = k;
    a.v = v;
    a.ks = (size_t)k_stride;
    a.vs = (size_t)v_stride;
    a.slots = slots;
    return ran(beam::launch_attn_prep(a, static_cast<hipStream_t>(stream)));
}

beam_status beam_moe_kv_read(const beam_moe_attn_cfg* cfg, int32_t B, int32_t N, const beam_moe_kv_cache* cache,
                             const int32_t* page_table, int32_t max_pages, const int32_t* row_offsets,
                             const int32_t* first, void* k_out, void* v_out, beam_dtype dtype, void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (B < 0 || B > kMaxT || N < 0 || N > beam::kMaxReadRows || max_pages < 0 || !act_dtype(dtype))
        return BEAM_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return BEAM_OK;
    if (!row_offsets || !aligned4(row_offsets) || !aligned4(first) || !k_out || !v_out || !aligned16(k_out) ||
        !aligned16(v_out))
        return BEAM_ERR_INVALID_ARG;
    const size_t ob = (size_t)N * cfg->n_kv_heads * cfg->head_dim * (dtype == BEAM_BF16 ? 2 : 4);
    if (overlap(k_out, ob, v_out, ob)) return BEAM_ERR_INVALID_ARG;
    if (max_pages > 0 && (!page_table || !aligned4(page_table))) return BEAM_ERR_INVALID_ARG;
    beam::KvReadArgs a{};
    st = check_cache(cfg, cache, a.c);
    if (st != BEAM_OK) return st;
    a.B = B;
    a.N = N;
    a.Hkv = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.max_pages = max_pages;
    a.bf16 = dtype == BEAM_BF16;
    a.table = page_table;
    a.offsets = row_offsets;
    a.first = first;
    a.k_out = k_out;
    a.v_out = v_out;
    return ran(beam::launch_kv_read(a, static_cast<hipStream_t>(stream)));
}

size_t beam_moe_attn_workspace_bytes(const beam_moe_attn_cfg* cfg, int32_t B, int32_t max_len) {
    return beam_moe_attn_decode_sinks_workspace_bytes(cfg, 0, B, max_len);
}

size_t beam_moe_attn_decode_sinks_workspace_bytes(const beam_moe_attn_cfg* cfg, int32_t n_sinks, int32_t B,
                                                  int32_t max_len) {
    if (check_attn_cfg(cfg) != BEAM_OK || B <= 0 || B > kMaxT || max_len < 0 || max_len > beam::kMaxLen ||
        !sinks_ok(n_sinks))
        return 0;
    return beam::attn_decode_ws_bytes(B, cfg->n_heads, cfg->head_dim,
                                      beam::attn_decode_split(B, cfg->n_kv_heads, max_len, cfg->window, n_sinks));
}

beam_status beam_moe_attn_decode(const beam_moe_attn_cfg* cfg, int32_t B, const void* q, int64_t q_stride,
                                 beam_dtype dtype, const beam_moe_kv_cache* cache, const int32_t* page_table,
                                 int32_t max_pages, const int32_t* seq_lens, int32_t max_len, void* out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
    return beam_moe_attn_decode_sinks(cfg, 0, B, q, q_stride, dtype, cache, page_table, max_pages, seq_lens, max_len,
                                      out, lse, ws, ws_bytes, stream);
}

beam_status beam_moe_attn_decode_sinks(const beam_moe_attn_cfg* cfg, int32_t n_sinks, int32_t B, const void* q,
                                       int64_t q_stride, beam_dtype dtype, const beam_moe_kv_cache* cache,
                                       const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                       int32_t max_len, void* out, float* lse, void* ws, size_t ws_bytes,
                                       void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (B < 0 || B > kMaxT || max_pages < 0 || max_len < 0 || max_len > beam::kMaxLen || !act_dtype(dtype) ||
        !sinks_ok(n_sinks))
        return BEAM_ERR_INVALID_ARG;
    if (B == 0) return BEAM_OK;
    const int64_t qw = (int64_t)cfg->n_heads * cfg->head_dim;
    if (!rows_ok(q, q_stride, qw) || !out || !aligned16(out) || !seq_lens || !aligned4(seq_lens) || !aligned4(lse))
        return BEAM_ERR_INVALID_ARG;
    if (max_pages > 0 && (!page_table || !aligned4(page_table))) return BEAM_ERR_INVALID_ARG;
    beam::AttnDecodeArgs a{};
    st = check_cache(cfg, cache, a.c);
    if (st != BEAM_OK) return st;
    if ((a.c.kind == beam::A_F32) != (dtype == BEAM_F32)) return BEAM_ERR_UNSUPPORTED;
    const size_t es = dtype == BEAM_BF16 ? 2 : 4;
    if (overlap(out, (size_t)B * qw * es, q, span_bytes(B, q_stride, qw, es))) return BEAM_ERR_INVALID_ARG;
    a.p = beam::attn_decode_split(B, cfg->n_kv_heads, max_len, cfg->window, n_sinks);
    if ((int64_t)a.p.rows * cfg->n_heads > kMaxParts) return BEAM_ERR_UNSUPPORTED;
    const size_t need = beam::attn_decode_ws_bytes(B, cfg->n_heads, cfg->head_dim, a.p);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return BEAM_ERR_WORKSPACE;
    a.B = B;
    a.Hq = cfg->n_heads;
    a.Hkv = cfg->n_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.D = cfg->head_dim;
    a.max_pages = max_pages;
    a.window = cfg->window;
    a.sinks = cfg->window > 0 ? n_sinks : 0;
    a.scale = cfg->softmax_scale;
    a.q = q;
    a.qs = (size_t)q_stride;
    a.table = page_table;
    a.lens = seq_lens;
    a.out = out;
    a.lse = lse;
    return ran(beam::launch_attn_decode(a, ws, static_cast<hipStream_t>(stream)));
}

// max_len counts in whole pages: so a workspace for the longest length serves a
// call that expects what its table holds
static beam::PromptSplit prompt_split(const beam_moe_attn_cfg& cfg, int32_t n_sinks, int32_t B, int32_t T,
                                      int32_t max_len) {
    const int32_t pages = (max_len + cfg.page_size - 1) & -cfg.page_size;   // at most kMaxLen, as max_len is
    return beam::attn_prompt_split(B, T, cfg.n_heads, cfg.n_kv_heads, pages, cfg.window, n_sinks);
}
size_t beam_moe_attn_prompt_workspace_bytes(const beam_moe_attn_cfg* cfg, int32_t n_sinks, int32_t B, int32_t T,
                                            int32_t max_len) {
    if (check_attn_cfg(cfg) != BEAM_OK || B <= 0 || B > kMaxT || T <= 0 || T > kMaxT || max_len < 0 ||
        max_len > beam::kMaxLen || !sinks_ok(n_sinks))
        return 0;
    return beam::attn_prompt_ws_bytes(cfg->n_kv_heads, cfg->head_dim, prompt_split(*cfg, n_sinks, B, T, max_len));
}

beam_status beam_moe_attn_prompt(const beam_moe_attn_cfg* cfg, int32_t n_sinks, int32_t B, int32_t T, const void* q,
                                 int64_t q_stride, beam_dtype dtype, const beam_moe_kv_cache* cache,
                                 const int32_t* page_table, int32_t max_pages, const int32_t* q_offsets,
                                 const int32_t* seq_lens, int32_t max_len, void* out, float* lse, void* ws,
                                 size_t ws_bytes, void* stream) {
    beam_status st = check_attn_cfg(cfg);
    if (st != BEAM_OK) return st;
    if (B < 0 || B > kMaxT || T < 0 || T > kMaxT || max_pages < 0 || max_len < 0 || max_len > beam::kMaxLen ||
        !act_dtype(dtype) || !sinks_ok(n_sinks))
        return BEAM_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return BEAM_OK;
    const int64_t qw = (int64_t)cfg->n_heads * cfg->head_dim;
    if (!rows_ok(q, q_stride, qw) || !out || !aligned16(out) || !seq_lens || !aligned4(seq_lens) || !q_offsets ||
        !aligned4(q_offsets) || !aligned4(lse))
        return BEAM_ERR_INVALID_ARG;
    if (max_pages > 0 && (!page_table || !aligned4(page_table))) return BEAM_ERR_INVALID_ARG;
    beam::AttnPromptArgs a{};
    st = check_cache(cfg, cache, a.c);
    if (st != BEAM_OK) return st;
    if ((a.c.kind == beam::A_F32) != (dtype == BEAM_F32)) return BEAM_ERR_UNSUPPORTED;
    const size_t es = dtype == BEAM_BF16 ? 2 : 4;
    if (overlap(out, (size_t)T * qw * es, q, span_bytes(T, q_stride, qw, es))) return BEAM_ERR_INVALID_ARG;
    a.p = prompt_split(*cfg, n_sinks, B, T, max_len);
    if (a.p.groups(cfg->n_kv_heads) >= kMaxGroups) return BEAM_ERR_UNSUPPORTED;
    const size_t need = beam::attn_prompt_ws_bytes(cfg->n_kv_heads, cfg->head_dim, a.p);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return BEAM_ERR_WORKSPACE;
    a.B = B;
    a.T = T;
    a.Hq = cfg->n_heads;
    a.Hkv = cfg->n_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.D = cfg->head_dim;
    a.max_pages = max_pages;
    a.window = cfg->window < beam::kMaxLen ? cfg->window : beam::kMaxLen;   // as far as any; differences of 32 bits hold it
    a.sinks = cfg->window > 0 ? n_sinks : 0;
    a.scale = cfg->softmax_scale;
    a.q = q;
    a.qs = (size_t)q_stride;
    a.table = page_table;
    a.offsets = q_offsets;
    a.lens = seq_lens;
    a.out = out;
    a.lse = lse;
    return ran(beam::launch_attn_prompt(a, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
