"""GPU parity of the attention sublayer's entry points against the fp64
oracle (oracle/attn.py): head layouts, odd sizes, lengths from none to many
parts, windows, bad pages, garbage in unwritten places, strides, streams,
captured graphs, and the calls chained as a decode step uses them.

Tolerances, from the arithmetic.  h(t) = finfo(t).eps / 2 is the relative
error of one rounding to t, u = h(fp32) = 2^-24.

Norm and rotation, per head row with largest magnitude M (after norm and
factor): the sum of D <= 256 squares (8 in a lane, then log2 steps), the
square root, the quotient and two products are each good to a few u (16 u in
all), the reduced angle is off by at most pi * u + 2 ulp of sin and cos (8 u),
a rotated element adds two such products of magnitude at most M and the
position factor 4 u more: below 64 u M = 2^-18 M, plus h(dtype) |value|.

Decode, with A = sum_j softmax_j |v_j| and Z = scale * max_j sum_d |q_d k_jd|:
a score's products are exact (bf16, e4m3) or off by u each, and summed in at
most D/4 + 8 steps, so it is off by e = (D/4 + 8) u Z, which moves a
probability by the factor 1 + 2 e; exp2, the rescalings and the n-term sums in
fp32 add (n/32 + 64) u; a probability is rounded to bf16 once (bf16 and e4m3
caches: h(bf16), and the value's scale, where there is one, enters before that
rounding, 2 u).  So out is off by
(h(bf16) or 0 + 2 e + (n/32 + 64) u) A + h(dtype) |out|, and lse by
e + (n/32 + 64) u + u |lse|.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import synth
from parity_util import say

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
KIND = {"f32": beam.BEAM_F32, "bf16": beam.BEAM_BF16, "fp8": beam.BEAM_FP8_E4M3}
ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return synth.to_f64(t.float() if t.dtype == torch.float8_e4m3fn else t)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def poisoned(cfg, n_pages, kind):
    """A cache whose every element is NaN."""
    c = beam.kv_cache(cfg, n_pages, KIND[kind], DEV)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            (t.view(torch.uint8).fill_(0x7F) if t.dtype == torch.float8_e4m3fn else t.fill_(float("nan")))
    return c


def filled(cfg, n_pages, kind, seed):
    """A cache of random rows, and its exact values k, v [n_pages, h, P, D]."""
    c = beam.kv_cache(cfg, n_pages, KIND[kind], DEV)
    g = gen(seed)
    vals = []
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = torch.randn(t.shape, generator=g, device=DEV)
        if kind == "fp8":
            s.copy_(x.abs().amax(-1) / 448)
            t.copy_((x / s[..., None]).to(torch.float8_e4m3fn))
            vals.append(f64(t) * f64(s)[..., None])
        else:
            t.copy_(x)
            vals.append(f64(t))
    return c, vals


# ------------------------------------------------------------------ norm, rotation, cache rows

def rope_inputs(cfg, T, act, seed, gap=0):
    """Columns of a merged projection (with `gap` columns before and between), positions, gammas, frequencies."""
    g = gen(seed)
    hq, hkv, D = cfg.n_heads, cfg.n_kv_heads, cfg.head_dim
    w = (hq + 2 * hkv) * D + 3 * gap
    m = torch.randn((T, w), generator=g, device=DEV).to(ACT[act])
    at = [gap, 2 * gap + hq * D, 3 * gap + (hq + hkv) * D]
    q, k, v = (m[:, a:a + h * D].unflatten(1, (h, D)) for a, h in zip(at, (hq, hkv, hkv)))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = (1 << 31) - 1, -7
    gq, gk = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(ACT[act]) for _ in range(2))
    f = None
    if cfg.rope_dim:
        f = (10000.0 ** (-torch.arange(0, cfg.rope_dim, 2, dtype=torch.float64) / cfg.rope_dim)).float().to(DEV)
    return q, k, v, pos, gq, gk, f


def rope_ref(cfg, x, gamma, pos, f, is_q):
    X, G, P = f64(x), None if gamma is None else f64(gamma), f64(pos)
    F = None if f is None else f64(f)
    return np.stack([np.stack([oracle.norm_rope_row(
        X[t, h], G, cfg.rms_eps, P[t], F, cfg.rope_interleaved,
        oracle.ssmax_factor(P[t], cfg.ssmax_len, cfg.ssmax_exp) if is_q else 1.0) for h in range(X.shape[1])])
        for t in range(X.shape[0])])


def check_rows(name, got, ref, half):
    top = np.abs(ref).max(-1, keepdims=True)
    err = np.abs(f64(got) - ref) - half * np.abs(ref) - 2.0 ** -18 * top
    say(f"  {name}: over the bound by {err.max():.2e}")
    assert (err <= 0).all(), name


ROPE = [
    # act, T, n_heads, n_kv_heads, D, R, interleaved, ssmax, gammas, gap
    ("bf16", 1, 48, 8, 128, 128, False, 0.0, True, 0),
    ("bf16", 37, 48, 8, 128, 128, False, 0.0, True, 8),
    ("bf16", 5, 48, 8, 128, 0, False, 2048.0, True, 0),
    ("f32", 9, 16, 4, 64, 32, True, 0.0, True, 16),
    ("f32", 3, 5, 5, 256, 256, False, 100.0, True, 8),
    ("bf16", 7, 3, 1, 64, 48, False, 0.0, False, 8),
    ("bf16", 4, 7, 7, 256, 16, True, 0.0, True, 0),
    ("f32", 130, 3, 1, 128, 64, False, 0.0, False, 0),
    ("bf16", 6, 2, 2, 256, 128, False, 0.0, True, 0),
    ("bf16", 6, 5, 1, 128, 96, False, 0.0, True, 0),
    ("f32", 4, 4, 2, 64, 64, False, 0.0, True, 0),
    ("bf16", 3, 2, 1, 256, 256, True, 0.0, True, 8),
    ("bf16", 2, 256, 4, 64, 32, False, 0.0, True, 0),
]


@pytest.mark.parametrize("act,T,hq,hkv,D,R,inter,ssmax,norm,gap", ROPE)
def test_qk_norm_rope(act, T, hq, hkv, D, R, inter, ssmax, norm, gap):
    say(f"qk_norm_rope {act} T={T} {hq}/{hkv} D={D} R={R}")
    cfg = beam.AttnCfg(hq, hkv, D, R, inter, 0, 16, ssmax)
    q, k, _, pos, gq, gk, f = rope_inputs(cfg, T, act, 3 + T, gap)
    if not norm:
        gq = gk = None
    qo = torch.full((T + 1, hq, D), 5.0, dtype=ACT[act], device=DEV)
    ko = torch.full((T + 1, hkv, D), 5.0, dtype=ACT[act], device=DEV)
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, qo[:T], ko[:T], f, gq, gk)
    torch.cuda.synchronize()
    check_rows("q", qo[:T], rope_ref(cfg, q, gq, pos, f, True), HALF[ACT[act]])
    check_rows("k", ko[:T], rope_ref(cfg, k, gk, pos, f, False), HALF[ACT[act]])
    assert (qo[T] == 5).all() and (ko[T] == 5).all()       # rows behind the last stay


def rope_torch(cfg, x, gamma, pos, f, is_q):
    """The formula over many tokens at once, in fp64 torch."""
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + cfg.rms_eps).sqrt() * gamma.double()
    if cfg.rope_dim:
        a = pos.double()[:, None, None] * f.double()
        half, y = cfg.rope_dim // 2, x.clone()
        iu, iw = (slice(0, cfg.rope_dim, 2), slice(1, cfg.rope_dim, 2)) if cfg.rope_interleaved else (
            slice(0, half), slice(half, cfg.rope_dim))
        y[..., iu] = x[..., iu] * a.cos() - x[..., iw] * a.sin()
        y[..., iw] = x[..., iw] * a.cos() + x[..., iu] * a.sin()
        x = y
    if is_q and cfg.ssmax_len:
        x = x * ((1 + pos.double().clamp(min=0) / cfg.ssmax_len) ** cfg.ssmax_exp)[:, None, None]
    return x


# many tokens: a wave then takes several groups of a token's heads, here 2, 3
# (of 16, so the last wave of a token has one), 2 with one group of queries,
# keys and values together, and all 4
@pytest.mark.parametrize("act,kind,T,hq,hkv,D,R,inter,ssmax", [
    ("bf16", "bf16", 5000, 48, 8, 128, 128, False, 0.0), ("bf16", "fp8", 7001, 48, 8, 128, 128, False, 0.0),
    ("f32", "f32", 33000, 9, 3, 64, 32, True, 0.0), ("bf16", "fp8", 40000, 4, 2, 256, 0, False, 2048.0),
])
def test_qk_norm_rope_many_tokens(act, kind, T, hq, hkv, D, R, inter, ssmax):
    say(f"many tokens {act} -> {kind} T={T} {hq}/{hkv} D={D}")
    cfg = beam.AttnCfg(hq, hkv, D, R, inter, 0, 64, ssmax)
    q, k, v, pos, gq, gk, f = rope_inputs(cfg, T, act, T)
    n_pages = T // 64 + 2
    slots = torch.randperm(n_pages * 64, generator=gen(1), device=DEV)[:T].to(torch.int32)
    c = beam.kv_cache(cfg, n_pages, KIND[kind], DEV)
    qo, q2 = (torch.empty((T, hq, D), dtype=ACT[act], device=DEV) for _ in range(2))
    ko = torch.empty((T, hkv, D), dtype=ACT[act], device=DEV)
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, qo, ko, f, gq, gk)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, q2, c, f, gq, gk)
    torch.cuda.synchronize()
    assert torch.equal(qo, q2)
    half = HALF[ACT[act]]
    rq, rk = rope_torch(cfg, q, gq, pos, f, True), rope_torch(cfg, k, gk, pos, f, False)
    for got, ref in ((qo, rq), (ko, rk)):
        top = ref.abs().amax(-1, keepdim=True)
        assert ((got.double() - ref).abs() <= half * ref.abs() + 2.0 ** -18 * top).all()
    at = (slots // 64).long(), slice(None), (slots % 64).long()
    for side, scale, ref in ((c.k, c.k_scale, rk), (c.v, c.v_scale, v.double())):
        got = side[at].double() if kind != "fp8" else side.view(torch.uint8)[at].view(
            torch.float8_e4m3fn).double() * scale[at].double()[..., None]
        top = ref.abs().amax(-1, keepdim=True)
        step = 2.0 ** -4 * ref.abs() + 2.0 ** -10 * top / 448 if kind == "fp8" else HALF[ACT[kind]] * ref.abs()
        assert ((got - ref).abs() <= step + 2.0 ** -17 * top).all()


def test_qk_norm_rope_in_place():
    cfg = beam.AttnCfg(6, 2, 128, 64)
    q, k, _, pos, gq, gk, f = rope_inputs(cfg, 19, "bf16", 5)
    q, k = q.contiguous(), k.contiguous()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, qo, ko, f, gq, gk)
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, q, k, f, gq, gk)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_norm_of_zeros_and_non_finite_rows():
    """A row of zeros stays zero; a non-finite element makes its own head row
    NaN (with the norm) or only its own pair (without), and no other."""
    cfg = beam.AttnCfg(4, 2, 64, 32)
    q, k, _, pos, gq, gk, f = rope_inputs(cfg, 4, "bf16", 6)
    q, k = q.contiguous(), k.contiguous()
    q[0, 1] = 0
    q[1, 2, 60] = float("inf")
    k[2, 0, 3] = float("nan")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, qo, ko, f, gq, gk)
    torch.cuda.synchronize()
    assert (qo[0, 1] == 0).all()
    bad = torch.isnan(qo).any(-1)
    assert bad.sum() == 1 and bad[1, 2]
    bad = torch.isnan(ko).any(-1)
    assert bad.sum() == 1 and bad[2, 0]
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, qo, ko, f)
    torch.cuda.synchronize()
    assert torch.isinf(qo[1, 2, 60]) and torch.isfinite(qo).sum() == qo.numel() - 1
    bad = torch.nonzero(~torch.isfinite(ko[2, 0]))[:, 0].tolist()
    assert bad == [3, 19] and torch.isfinite(ko).sum() == ko.numel() - 2


def stored(c, slots, cfg):
    """fp64 values, and scales, of the cache rows [len(slots), h, D] at slots."""
    s = torch.as_tensor(slots, device=DEV).long()
    at = s // cfg.page_size, slice(None), s % cfg.page_size
    out = []
    for t, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        out.append((f64(t[at]), None if sc is None else f64(sc[at])))
    return out


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("act,T,hq,hkv,D,R,inter,ssmax,norm,gap", ROPE)
def test_qk_norm_rope_cache(kind, act, T, hq, hkv, D, R, inter, ssmax, norm, gap):
    say(f"qk_norm_rope_cache {act} -> {kind} T={T} {hq}/{hkv} D={D} R={R}")
    cfg = beam.AttnCfg(hq, hkv, D, R, inter, 0, 16, ssmax)
    q, k, v, pos, gq, gk, f = rope_inputs(cfg, T, act, 3 + T, gap)
    if not norm:
        gq = gk = None
    n_pages = T // 16 + 3
    slots = torch.randperm(n_pages * 16, generator=gen(T), device=DEV)[:T].to(torch.int32)
    if T > 4:                                   # rows that go nowhere
        slots[1], slots[3], slots[4] = -1, n_pages * 16, (1 << 31) - 1
    keep = ((slots >= 0) & (slots < n_pages * 16)).cpu().numpy()
    c = poisoned(cfg, n_pages, kind)
    qo = torch.empty((T, hq, D), dtype=ACT[act], device=DEV)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, qo, c, f, gq, gk)
    torch.cuda.synchronize()
    check_rows("q", qo, rope_ref(cfg, q, gq, pos, f, True), HALF[ACT[act]])
    (gotk, ks), (gotv, vs) = stored(c, slots.cpu().numpy()[keep], cfg)
    refk, refv = rope_ref(cfg, k, gk, pos, f, False)[keep], f64(v)[keep]
    if kind == "fp8":
        # the scale follows the row's maximum; a code is off by half a step of
        # its binade (2^-4 relative) or of the smallest one (2^-10 scales)
        top = np.abs(refk).max(-1)
        assert (np.abs(ks - top / 448) <= 2.0 ** -17 * top / 448).all()
        err = np.abs(gotk * ks[..., None] - refk)
        assert (err <= 2.0 ** -4 * np.abs(refk) + 2.0 ** -10 * ks[..., None] + 2.0 ** -17 * top[..., None]).all()
        for t in range(len(refv)):              # values: the oracle's codes, bit for bit
            for h in range(hkv):
                sc, codes = oracle.quantize_row_e4m3(refv[t, h])
                assert sc == vs[t, h] and np.array_equal(codes, gotv[t, h])
    else:
        half = HALF[ACT[kind]]
        top = np.abs(refk).max(-1, keepdims=True)
        assert (np.abs(gotk - refk) <= half * np.abs(refk) + 2.0 ** -18 * top).all()
        assert np.array_equal(gotv, refv if act == "bf16" or kind == "f32" else oracle.round_bf16(refv))
    # nothing else in the cache was touched
    untouched = np.setdiff1d(np.arange(n_pages * 16), slots.cpu().numpy()[keep])
    for got, sc in stored(c, untouched, cfg):
        assert np.isnan(got).all() and (sc is None or np.isnan(sc).all())


@pytest.mark.parametrize("act,kind,T,hkv,D,P", [
    ("bf16", "bf16", 33, 8, 128, 64), ("bf16", "fp8", 33, 8, 128, 16), ("f32", "fp8", 5, 3, 64, 32),
    ("f32", "f32", 1, 1, 256, 1024), ("bf16", "f32", 4, 2, 64, 128), ("f32", "bf16", 300, 1, 128, 16),
    ("bf16", "fp8", 1000, 5, 256, 64),
])
def test_kv_write_then_read(act, kind, T, hkv, D, P):
    """Written rows come back, bit for bit where the formats allow it; other
    slots stay; the rows are read in runs that begin and end inside pages."""
    say(f"kv write/read {act} {kind} T={T} hkv={hkv} D={D} P={P}")
    cfg = beam.AttnCfg(hkv, hkv, D, 0, False, 0, P)
    g = gen(T)
    m = torch.randn((T, 2 * hkv * D + 8), generator=g, device=DEV).to(ACT[act])
    k, v = m[:, :hkv * D].unflatten(1, (hkv, D)), m[:, hkv * D + 8:].unflatten(1, (hkv, D))
    k[0, 0] = 0                                            # an all-zero row: scale 1, codes 0
    # two sequences that share nothing, tokens in order, pages in any order
    n1 = T // 3
    lens = [n1, T - n1]
    width = -(-max(lens) // P) + 1
    n_pages = 2 * width + 1
    perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    table = np.full((3, width), -1, np.int32)
    slots = []
    for b, n in enumerate(lens):
        for j in range(-(-n // P)):
            table[b, j] = perm.pop()
        slots += [table[b, t // P] * P + t % P for t in range(n)]
    c = poisoned(cfg, n_pages, kind)
    beam.beam_moe_kv_write(cfg, k, v, torch.tensor(slots, dtype=torch.int32, device=DEV), c)
    torch.cuda.synchronize()
    ref = []
    for x, (got, sc) in zip((f64(k), f64(v)), stored(c, slots, cfg)):
        if kind == "fp8":
            want = np.zeros_like(x)
            for t in range(T):
                for h in range(hkv):
                    s, codes = oracle.quantize_row_e4m3(x[t, h])
                    assert s == sc[t, h] and np.array_equal(codes, got[t, h])
                    want[t, h] = codes * s
        else:
            want = oracle.round_bf16(x) if kind == "bf16" else x
            assert np.array_equal(got, want)
        ref.append(want)
    free = np.setdiff1d(np.arange(n_pages * P), slots)
    for got, sc in stored(c, free, cfg):
        assert np.isnan(got).all() and (sc is None or np.isnan(sc).all())

    # runs: from inside the first sequence, all of the second, none of the third
    first = [n1 // 2, 0, 0]
    off = np.cumsum([0, n1 - n1 // 2, T - n1, 0]).astype(np.int32)
    rows = [t for t in range(n1 // 2, n1)] + [t for t in range(n1, T)]
    table = torch.tensor(table, device=DEV)
    for out in ("bf16", "f32"):
        ko, vo = (torch.full((len(rows) + 3, hkv, D), 7.0, dtype=ACT[out], device=DEV) for _ in range(2))
        beam.beam_moe_kv_read(cfg, c, table, torch.tensor(off, device=DEV), ko, vo,
                              first=torch.tensor(first, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        for got, want in ((ko, ref[0]), (vo, ref[1])):
            want = want[rows].astype(np.float32).astype(np.float64)     # code * scale in fp32
            assert np.array_equal(f64(got[:len(rows)]), want if out == "f32" else oracle.round_bf16(want))
            assert (got[len(rows):] == 7).all()


def test_codes_as_bytes():
    """A cache of uint8 codes is the same cache as one of float8_e4m3fn."""
    cfg = beam.AttnCfg(4, 2, 64, 0, False, 0, 16)
    c, _ = filled(cfg, 4, "fp8", 3)
    b = beam.KVCache(c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)
    t = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 4, 64), generator=gen(1), device=DEV).bfloat16()
    outs = []
    for x in (c, b):
        o = torch.empty_like(q)
        beam.beam_moe_attn_decode(cfg, q, x, t, torch.tensor([40], dtype=torch.int32, device=DEV), 40, o, None)
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(*outs)


def test_every_code_is_exact():
    """All 256 e4m3 codes through both readers: the row of one seen token is
    the decode's result (its probability is 1), NaN codes included."""
    cfg = beam.AttnCfg(2, 2, 128, 0, False, 0, 16)
    c = beam.kv_cache(cfg, 1, beam.BEAM_FP8_E4M3, DEV)
    c.k.view(torch.uint8).zero_()
    codes = torch.arange(256, device=DEV, dtype=torch.int32).to(torch.uint8).view(2, 128)
    c.v.view(torch.uint8)[0, :, 0] = codes
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    t = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    beam.beam_moe_attn_decode(cfg, q, c, t, one, 1, out, None)
    ko, vo = (torch.empty((1, 2, 128), device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, t, torch.tensor([0, 1], dtype=torch.int32, device=DEV), ko, vo)
    torch.cuda.synchronize()
    want = oracle.e4m3_decode(codes.cpu().numpy())
    for got in (out, vo):
        assert np.array_equal(f64(got)[0], want, equal_nan=True)


@pytest.mark.parametrize("B,every", [(3, 1), (64, 1), (65, 1), (700, 1), (700, 150), (9000, 1), (9000, 400)])
def test_kv_read_empty_sequences_between(B, every):
    """Sequences without rows at the front, in the middle and at the end, and
    many sequences; long runs of empty ones inside a workgroup's rows."""
    cfg = beam.AttnCfg(3, 3, 64, 0, False, 0, 16)
    g = np.random.default_rng(1)
    n = g.integers(0, 4, B) * g.integers(0, 12, B) if every == 1 else np.where(np.arange(B) % every == 7, 3, 0)
    n[1] = 40
    n[0], n[-1] = 0, 0
    c, (k, v) = filled(cfg, 50, "bf16", 2)
    table = g.integers(0, 50, (B, 3)).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N = int(off[-1])
    ko, vo = (torch.empty((N, 3, 64), device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, torch.tensor(table, device=DEV), torch.tensor(off, device=DEV), ko, vo)
    torch.cuda.synchronize()
    b = np.repeat(np.arange(B), n)
    t = np.arange(N) - off[b]
    for got, ref in ((ko, k), (vo, v)):
        assert np.array_equal(f64(got), ref[table[b, t // 16], :, t % 16])


def test_kv_read_outside_the_cache():
    """Bad pages, tokens before the first and behind the table read as zeros."""
    cfg = beam.AttnCfg(2, 2, 64, 0, False, 0, 16)
    c, (k, _) = filled(cfg, 3, "fp8", 1)
    table = torch.tensor([[0, -1, 3], [1 << 30, 2, -(1 << 31)], [1, 1, 1]], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 60, 80, 90], dtype=torch.int32, device=DEV)
    first = torch.tensor([0, 10, -5], dtype=torch.int32, device=DEV)
    ko, vo = (torch.full((90, 2, 64), 3.0, device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, table, off, ko, vo, first=first)
    torch.cuda.synchronize()
    want = np.zeros((90, 2, 64))
    for i in range(90):
        b, t = (0, i) if i < 60 else (1, 10 + i - 60) if i < 80 else (2, i - 80 - 5)
        p = table[b, t // 16].item() if 0 <= t < 48 else -1
        if 0 <= p < 3:
            want[i] = k[p, :, t % 16]
    assert np.array_equal(f64(ko), want.astype(np.float32).astype(np.float64))


# ------------------------------------------------------------------ decode

def tables(lens, P, n_pages, seed, width=None):
    """A page table of distinct random pages, -1 behind each sequence."""
    width = width or max(1, -(-max(lens) // P))
    perm = np.random.default_rng(seed).permutation(n_pages).tolist()
    t = np.full((len(lens), width), -1, np.int32)
    for b, n in enumerate(lens):
        for j in range(min(width, -(-n // P))):
            t[b, j] = perm.pop()
    return t


def decode_ref(cfg, q, k, v, table, lens, n_pages):
    """(out, lse, bound on out, bound on lse) of every sequence."""
    B, hq, D = q.shape
    hkv = cfg.n_kv_heads
    P, act = cfg.page_size, q.dtype
    out, lse = np.zeros((B, hq, D)), np.zeros((B, hq))
    eo, el = np.zeros((B, hq, D)), np.zeros((B, hq))
    for b, n in enumerate(lens):
        n = min(max(n, 0), table.shape[1] * P)
        toks = range(max(0, n - cfg.window) if cfg.window else 0, n)
        kr, there = oracle.cached_rows(k, table[b], toks, n_pages)
        vr, _ = oracle.cached_rows(v, table[b], toks, n_pages)
        kr, vr = kr[there], vr[there]
        qb = f64(q[b]).reshape(hkv, hq // hkv, D)
        o, z, mag = oracle.decode_attention(qb, kr, vr, cfg.softmax_scale)
        Z = 0.0
        if len(kr):
            Z = cfg.softmax_scale * max((np.abs(qb[h]) @ np.abs(kr[:, h]).T).max() for h in range(hkv))
        e = (D / 4 + 8) * U * Z
        c = len(kr) / 32 + 64
        half_p = 0.0 if act == torch.float32 else 2.0 ** -8 + 2 * U
        out[b], lse[b] = o.reshape(hq, D), z.reshape(hq)
        eo[b] = (half_p + 2 * e + c * U) * mag.reshape(hq, D) + HALF[act] * np.abs(out[b])
        el[b] = e + c * U + U * np.abs(np.where(np.isinf(lse[b]), 0, lse[b]))
    return out, lse, eo, el


def check_decode(cfg, q, c, vals, table, lens, max_len, name, n_pages=None, stream=None):
    n_pages = n_pages or c.k.shape[0]
    B = len(lens)
    dt = torch.tensor(table, device=DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)     # dense, whatever q's rows are
    lse = torch.full((B, cfg.n_heads), 9.0, device=DEV)
    ws = beam.attn_workspace(cfg, B, max_len)
    ws.view(torch.uint8).fill_(0xFF)                       # its contents do not matter
    beam.beam_moe_attn_decode(cfg, q, c, dt, dl, max_len, out, ws, lse)
    torch.cuda.synchronize()
    ro, rl, eo, el = decode_ref(cfg, q, *vals, table, lens, n_pages)
    got, gl = f64(out), f64(lse)
    d = np.abs(got - ro) - eo
    inf = np.isinf(rl)
    say(f"  {name}: out over the bound by {d.max():.2e}, lse max err {np.abs(np.where(inf, 0, gl - np.where(inf, 0, rl))).max():.2e}")
    assert (d <= 0).all(), name
    assert (got[np.broadcast_to(inf[..., None], got.shape)] == 0).all()
    assert np.array_equal(np.isneginf(gl), inf) and (np.abs(gl[~inf] - rl[~inf]) <= el[~inf]).all(), name
    return out


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 300, 513]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(48, 8, 128), (4, 4, 64), (16, 1, 256), (17, 1, 128), (48, 1, 64), (64, 1, 128),
                                      (40, 2, 256), (6, 2, 64)])
@pytest.mark.parametrize("window,P", [(0, 16), (100, 64)])
def test_decode(kind, hq, hkv, D, window, P):
    say(f"decode {kind} {hq}/{hkv} D={D} window={window} P={P}")
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5)
    n_pages = sum(-(-n // P) for n in LENS) + 2
    c, vals = filled(cfg, n_pages, kind, 7)
    table = tables(LENS, P, n_pages, 1)
    q = torch.randn((len(LENS), hq, D), generator=gen(2), device=DEV) * 2
    check_decode(cfg, q.to(ACT["f32" if kind == "f32" else "bf16"]), c, vals, table, LENS, max(LENS), "decode")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 512, 5000])
def test_decode_windows_and_garbage(kind, window):
    """Windows that begin anywhere in a page, NaN in every place that no
    query may see: behind the length, before the window, in free pages."""
    say(f"decode window {window} {kind}")
    lens = [1, 16, 47, 64, 65, 515, 640, 700]
    P = 64
    cfg = beam.AttnCfg(8, 2, 128, 0, False, window, P)
    n_pages = sum(-(-n // P) for n in lens) + 3
    c, vals = filled(cfg, n_pages, kind, 11)
    table = tables(lens, P, n_pages, 3)
    seen = np.zeros((n_pages, P), bool)
    for b, n in enumerate(lens):
        for t in range(max(0, n - window), n):
            seen[table[b, t // P], t % P] = True
    hide = torch.tensor(~seen, device=DEV)[:, None, :].expand(n_pages, 2, P)
    for t in (c.k, c.v):
        if kind == "fp8":
            t.view(torch.uint8)[hide] = 0x7F
        else:
            t[hide] = float("nan")
    for s in (c.k_scale, c.v_scale):
        if s is not None:
            s[hide] = float("nan")
    q = torch.randn((len(lens), 8, 128), generator=gen(4), device=DEV)
    check_decode(cfg, q.to(ACT["f32" if kind == "f32" else "bf16"]), c, vals, table, lens, max(lens), "window")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_decode_bad_pages_and_lengths(kind):
    """Pages outside the cache are skipped (also all of them), lengths below
    zero count as zero and beyond the table as the table's."""
    P, n_pages = 16, 12
    cfg = beam.AttnCfg(6, 2, 64, 0, False, 0, P)
    c, vals = filled(cfg, n_pages, kind, 5)
    table = np.array([[0, -1, 2, 3], [n_pages, 4, 1 << 30, 5], [-1, -1, -1, -1], [6, 7, 8, 9], [10, 11, 0, 1],
                      [-(1 << 31), 3, n_pages + 1, n_pages]], np.int32)
    lens = [60, 64, 33, -5, 1000, 49]
    q = torch.randn((6, 6, 64), generator=gen(4), device=DEV).to(ACT["f32" if kind == "f32" else "bf16"])
    check_decode(cfg, q, c, vals, table, lens, 64, "bad pages")


def test_decode_no_pages_at_all():
    cfg = beam.AttnCfg(6, 2, 64, 0, False, 0, 16)
    c, vals = filled(cfg, 1, "bf16", 5)
    q = torch.randn((3, 6, 64), generator=gen(4), device=DEV).bfloat16()
    check_decode(cfg, q, c, vals, np.zeros((3, 0), np.int32), [5, 0, 9], 100, "empty table")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("B,lens,max_len,window", [
    (1, [5000], 5000, 0),              # many parts
    (1, [5000], 100, 0),               # longer than expected
    (1, [40], 100000, 0),              # far shorter than expected
    (3, [4097, 0, 130], 4097, 0),
    (2, [3000, 2999], 4000, 1025),
    (5, [2048, 1, 700, 128, 1500], 2048, 0),
])
def test_decode_parts(kind, B, lens, max_len, window):
    say(f"decode parts {kind} {lens} expected {max_len} window {window}")
    P = 32
    cfg = beam.AttnCfg(6, 2, 128, 0, False, window, P)
    n_pages = sum(-(-n // P) for n in lens) + 1
    c, vals = filled(cfg, n_pages, kind, 9)
    q = torch.randn((B, 6, 128), generator=gen(6), device=DEV) * 3
    check_decode(cfg, q.to(ACT["f32" if kind == "f32" else "bf16"]), c, vals, tables(lens, P, n_pages, 2), lens,
                 max_len, "parts")


def test_decode_many_sequences_strided_queries():
    """Thousands of short sequences sharing pages, the largest page size, and
    queries that are columns of a wider matrix."""
    B, P, n_pages = 3000, 1024, 5
    cfg = beam.AttnCfg(6, 3, 64, 0, False, 0, P, softmax_scale=0.125)
    c, vals = filled(cfg, n_pages, "fp8", 4)
    g = np.random.default_rng(3)
    lens = g.integers(0, 40, B).tolist()
    table = g.integers(0, n_pages, (B, 1)).astype(np.int32)
    wide = torch.randn((B, 12 * 64), generator=gen(5), device=DEV).bfloat16()
    q = wide[:, 64:7 * 64].unflatten(1, (6, 64))
    check_decode(cfg, q, c, vals, table, lens, 40, "many sequences")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_decode_scores_far_apart(kind):
    """Scores that grow and fall by hundreds along the sequence: late maxima
    rescale what came before, early ones leave what follows at nothing."""
    P, lens = 16, [900, 900, 260]
    cfg = beam.AttnCfg(6, 2, 64, 0, False, 0, P, softmax_scale=1.0)
    n_pages = 140
    c = beam.kv_cache(cfg, n_pages, KIND[kind], DEV)
    table = tables(lens, P, n_pages, 8)
    g = gen(3)
    kk = torch.randn((n_pages, 2, P, 64), generator=g, device=DEV) * 0.1
    vv = torch.randn((n_pages, 2, P, 64), generator=g, device=DEV)
    for b, n in enumerate(lens):
        for t in range(n):
            up = t if b == 0 else n - t if b == 1 else (t * 37) % n
            kk[table[b, t // P], :, t % P, 0] = 0.5 * up
    vals = []
    for t, s, x in ((c.k, c.k_scale, kk), (c.v, c.v_scale, vv)):
        if kind == "fp8":
            s.copy_(x.abs().amax(-1) / 448)
            t.copy_((x / s[..., None]).to(torch.float8_e4m3fn))
            vals.append(f64(t) * f64(s)[..., None])
        else:
            t.copy_(x)
            vals.append(f64(t))
    q = torch.zeros((3, 6, 64), device=DEV)
    q[..., 0] = torch.tensor([1.0, -1.0, 0.25, 0.01, 2.0, -0.5], device=DEV)
    check_decode(cfg, q.to(ACT["f32" if kind == "f32" else "bf16"]), c, vals, table, lens, 900, "far apart")


def test_decode_non_finite():
    """A NaN or +inf key that is seen makes its heads NaN and no others; -inf
    scores count as nothing, all of them give an empty row."""
    P = 16
    cfg = beam.AttnCfg(4, 2, 64, 0, False, 0, P, softmax_scale=1.0)
    c, _ = filled(cfg, 9, "bf16", 5)
    table = torch.arange(9, dtype=torch.int32, device=DEV).view(3, 3)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    c.k[0, 0, 5, 7] = float("nan")          # sequence 0, kv head 0
    c.k[3:6, 1, :, 0] = float("-inf")       # sequence 1, kv head 1: every score -inf
    c.k[6, 0, 2, 0] = float("-inf")         # sequence 2, kv head 0: one of them
    out, lse = torch.empty_like(q), torch.empty((3, 4), device=DEV)
    for ml in (48, 4000):
        beam.beam_moe_attn_decode(cfg, q, c, table, torch.tensor([40, 48, 33], dtype=torch.int32, device=DEV), ml, out,
                                  beam.attn_workspace(cfg, 3, ml), lse)
        torch.cuda.synchronize()
        assert torch.isnan(out[0, :2]).all() and torch.isfinite(out[0, 2:]).all()
        assert (out[1, 2:] == 0).all() and torch.isneginf(lse[1, 2:]).all() and torch.isfinite(out[1, :2]).all()
        assert torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_offsets_beyond_32_bits(kind):
    """Pages whose elements lie past 2^31 (and bytes past 2^32) in the cache."""
    cfg = beam.AttnCfg(16, 8, 128, 128, False, 0, 64)
    n_pages = 40000                           # 64 * 1024 elements a page
    c = beam.kv_cache(cfg, n_pages, KIND[kind], DEV)
    T = 100
    pages = [39999, 33000]
    q, k, v, pos, gq, gk, f = rope_inputs(cfg, T, "bf16", 21)
    slots = torch.tensor([pages[t // 64] * 64 + t % 64 for t in range(T)], dtype=torch.int32, device=DEV)
    qo = torch.empty((T, 16, 128), dtype=torch.bfloat16, device=DEV)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, qo, c, f, gq, gk)
    small = beam.kv_cache(cfg, 2, KIND[kind], DEV)
    near = torch.arange(T, dtype=torch.int32, device=DEV)
    q2 = torch.empty_like(qo)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, near, q2, small, f, gq, gk)
    res = []
    for cache, tab in ((c, pages), (small, [0, 1])):
        table = torch.tensor([tab], dtype=torch.int32, device=DEV)
        ko, vo = (torch.empty((T, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        beam.beam_moe_kv_read(cfg, cache, table, torch.tensor([0, T], dtype=torch.int32, device=DEV), ko, vo)
        out = torch.empty((1, 16, 128), dtype=torch.bfloat16, device=DEV)
        beam.beam_moe_attn_decode(cfg, qo[-1:], cache, table, torch.tensor([T], dtype=torch.int32, device=DEV), T, out,
                                  beam.attn_workspace(cfg, 1, T))
        res.append((ko, vo, out))
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, b)


# ------------------------------------------------------------------ as it is used

def step_state(kind, B=6, P=16, seed=0):
    cfg = beam.AttnCfg(8, 2, 128, 128, False, 0, P)
    lens0 = [3, 0, 15, 16, 200, 640][:B]
    width, steps = 64, 4
    n_pages = sum(-(-(n + steps) // P) for n in lens0) + 1
    table = tables([n + steps for n in lens0], P, n_pages, seed, width)
    c, _ = filled(cfg, n_pages, kind, seed + 1)
    g = gen(seed + 2)
    qkv = torch.randn((steps, B, 12 * 128), generator=g, device=DEV).bfloat16()
    gq, gk = ((1 + 0.1 * torch.randn(128, generator=g, device=DEV)).bfloat16() for _ in range(2))
    f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().to(DEV)
    pos = torch.tensor([[n + s for n in lens0] for s in range(steps)], dtype=torch.int32, device=DEV)
    slots = torch.tensor([[table[b, (n + s) // P] * P + (n + s) % P for b, n in enumerate(lens0)]
                          for s in range(steps)], dtype=torch.int32, device=DEV)
    return cfg, table, c, qkv, gq, gk, f, pos, slots


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decode_steps(kind):
    """Steps of a decode loop, each attending to what the steps before it
    wrote; also as one captured graph replayed per step, and on another
    stream, with the same results."""
    cfg, table, c, qkv, gq, gk, f, pos, slots = step_state(kind)
    steps, B = qkv.shape[:2]
    bufs = beam.attn_buffers(cfg, B, 1024, keep_lse=True)
    t = torch.tensor(table, device=DEV)
    before = [x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]
    eager = []
    for s in range(steps):
        beam.attn_layer(cfg, qkv[s], pos[s], slots[s], c, t, pos[s] + 1, 1024, bufs, f, gq, gk)
        torch.cuda.synchronize()
        vals = []
        for x, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
            vals.append(f64(x) if sc is None else f64(x) * f64(sc)[..., None])
        lens = (pos[s] + 1).tolist()
        ro, rl, eo, el = decode_ref(cfg, bufs.q, *vals, table, lens, c.k.shape[0])
        assert (np.abs(f64(bufs.out) - ro) <= eo).all() and (np.abs(f64(bufs.lse) - rl) <= el).all()
        eager.append((bufs.out.clone(), bufs.lse.clone()))
    after = [x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]

    def rewind():
        for x, y in zip((x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None), before):
            x.copy_(y)

    inp, p, sl, ln = qkv[0].clone(), pos[0].clone(), slots[0].clone(), pos[0] + 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rewind()
        for s in range(steps):
            beam.attn_layer(cfg, qkv[s], pos[s], slots[s], c, t, pos[s] + 1, 1024, bufs, f, gq, gk)
            assert bufs.out is not None
            got = bufs.out.clone()
            side.synchronize()
            assert torch.equal(got, eager[s][0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beam.attn_layer(cfg, inp, p, sl, c, t, ln, 1024, bufs, f, gq, gk)
    for again in range(2):
        rewind()
        for s in range(steps):
            inp.copy_(qkv[s])
            p.copy_(pos[s])
            sl.copy_(slots[s])
            ln.copy_(pos[s] + 1)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(bufs.out, eager[s][0]) and torch.equal(bufs.lse, eager[s][1])
        for x, y in zip((x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None), after):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_decodes_at_once():
    """Two calls on two streams with a workspace each."""
    cfg = beam.AttnCfg(6, 2, 128, 0, False, 0, 32)
    lens = [3000, 1700]
    c, _ = filled(cfg, 160, "bf16", 9)
    t = torch.tensor(tables(lens, 32, 160, 2), device=DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [torch.randn((2, 6, 128), generator=gen(i), device=DEV).bfloat16() for i in range(2)]
    alone = []
    for q in qs:
        o = torch.empty_like(q)
        beam.beam_moe_attn_decode(cfg, q, c, t, n, 3000, o, beam.attn_workspace(cfg, 2, 3000))
        alone.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    ws = [beam.attn_workspace(cfg, 2, 3000) for _ in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, w, st in zip(qs, outs, ws, streams):
            beam.beam_moe_attn_decode(cfg, q, c, t, n, 3000, o, w, stream=st)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


def test_attention_between_two_boundaries():
    """One decode step of a small decoder layer: projection, attention,
    output projection, norm boundary, then the MoE layer on its x_next."""
    H, hq, hkv, D = 512, 4, 2, 128
    acfg = beam.AttnCfg(hq, hkv, D, 128, False, 512, 16)
    cfg = beam.LayerCfg(hidden=H, n_experts=16, n_groups=4, topk_groups=2, topk=4, group_topn=2, d_ff=256)
    g = gen(1)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)
    lens = [1, 40, 600]
    B, P = 3, 16
    n_pages = sum(-(-n // P) for n in lens) + 1
    table = tables(lens, P, n_pages, 4)
    c, _ = filled(acfg, n_pages, "fp8", 2)
    x, h = rnd(B, H).bfloat16(), rnd(B, H).bfloat16()
    wqkv, wo = rnd(8 * D, H) / math.sqrt(H), rnd(H, hq * D) / math.sqrt(hq * D)
    one = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    gq = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(DEV)
    pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
    slots = torch.tensor([table[b, (n - 1) // P] * P + (n - 1) % P for b, n in enumerate(lens)], dtype=torch.int32,
                         device=DEV)
    qkv = (x.float() @ wqkv.T).bfloat16()
    bufs = beam.attn_buffers(acfg, B, 1024)
    beam.attn_layer(acfg, qkv, pos, slots, c, torch.tensor(table, device=DEV), pos + 1, 1024, bufs, f, gq, gq)
    m = (bufs.out.float().view(B, -1) @ wo.T).contiguous()
    h0 = h.clone()
    xn = torch.empty_like(h)
    beam.beam_moe_norm_boundary(cfg, m, h, xn, one, one, 2)
    torch.cuda.synchronize()
    vals = [f64(t) * f64(s)[..., None] for t, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
    ro, _, eo, _ = decode_ref(acfg, bufs.q, *vals, table, lens, n_pages)
    assert (np.abs(f64(bufs.out) - ro) <= eo).all()
    # p, h' and x_next are rounded to bf16 one after the other: each may land one
    # step (2^-7 relative) off the oracle's, and carries the step before it on
    for b in range(B):
        rp, rh, rx = oracle.norm_boundary(f64(m)[b], f64(h0)[b], f64(one), f64(one), 2, cfg.rms_eps)
        size = np.abs(rp) + np.abs(f64(h0)[b])
        assert (np.abs(f64(h)[b] - rh) <= 2.0 ** -6 * (size + np.abs(rh))).all()
        assert (np.abs(f64(xn)[b] - rx) <= 2.0 ** -6 * (2 * size + np.abs(rx))).all()
    # the MoE layer takes x_next
    wr, bias = rnd(16, H) / math.sqrt(H), 28 + 0.02 * rnd(16)
    wgu, wd = (rnd(16, 512, H) / math.sqrt(H)).bfloat16(), (rnd(16, H, 256) / 16).bfloat16()
    pgu, pd = torch.empty_like(wgu), torch.empty_like(wd)
    beam.beam_moe_pack_weights(cfg, wgu, wd, pgu, pd)
    mb = beam.alloc_buffers(cfg, B, torch.bfloat16, beam.BEAM_BF16)
    beam.moe_layer(cfg, xn, wr, bias, pgu, pd, h, one, one, 3, mb)
    torch.cuda.synchronize()
    assert torch.isfinite(mb.x_next).all()


# ------------------------------------------------------------------ the binding

def binding_state():
    cfg = beam.AttnCfg(6, 2, 64, 32, False, 0, 16)
    q, k, v, pos, gq, gk, f = rope_inputs(cfg, 5, "bf16", 3, 8)
    c, _ = filled(cfg, 4, "fp8", 1)
    slots = torch.arange(5, dtype=torch.int32, device=DEV)
    return dict(
        cfg=cfg, q=q, k=k, v=v, pos=pos, gq=gq, gk=gk, f=f, cache=c, slots=slots,
        qo=torch.empty((5, 6, 64), dtype=torch.bfloat16, device=DEV),
        ko=torch.empty((5, 2, 64), dtype=torch.bfloat16, device=DEV),
        kr=torch.empty((7, 2, 64), dtype=torch.bfloat16, device=DEV),
        vr=torch.empty((7, 2, 64), dtype=torch.bfloat16, device=DEV),
        table=torch.tensor([[0, 1], [2, 3], [1, 2], [3, 0], [0, 0]], dtype=torch.int32, device=DEV),
        off=torch.tensor([0, 3, 3, 7, 7, 7], dtype=torch.int32, device=DEV),
        first=torch.tensor([2, 0, 20, 0, 0], dtype=torch.int32, device=DEV),
        lens=torch.tensor([9, 32, 0, 17, 1], dtype=torch.int32, device=DEV),
        out=torch.empty((5, 6, 64), dtype=torch.bfloat16, device=DEV), lse=torch.empty((5, 6), device=DEV),
        ws=beam.attn_workspace(cfg, 5, 32))


CALLS = {
    "rope": lambda s, **kw: beam.beam_moe_qk_norm_rope(s["cfg"], s["q"], s["k"], s["pos"], s["qo"], s["ko"], s["f"],
                                                       s["gq"], s["gk"], **kw),
    "rope_cache": lambda s, **kw: beam.beam_moe_qk_norm_rope_cache(
        s["cfg"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["qo"], s["cache"], s["f"], s["gq"], s["gk"], **kw),
    "write": lambda s, **kw: beam.beam_moe_kv_write(s["cfg"], s["k"], s["v"], s["slots"], s["cache"], **kw),
    "read": lambda s, **kw: beam.beam_moe_kv_read(s["cfg"], s["cache"], s["table"], s["off"], s["kr"], s["vr"],
                                                  first=s["first"], **kw),
    "decode": lambda s, **kw: beam.beam_moe_attn_decode(s["cfg"], s["qo"], s["cache"], s["table"], s["lens"], 32,
                                                        s["out"], s["ws"], s["lse"], **kw),
}
RESULTS = {"rope": ("qo", "ko"), "rope_cache": ("qo",), "write": (), "read": ("kr", "vr"), "decode": ("out", "lse")}


@pytest.mark.parametrize("name", CALLS)
def test_native_marshalling_is_the_python_one(name, monkeypatch):
    """A good call goes through the native marshalling, parameters that
    require gradients and tensors without a slope in their strides too, and
    does what the Python one does (taken with an explicit stream)."""
    s = binding_state()
    s["qo"].copy_(s["q"])
    s["gq"], s["f"] = torch.nn.Parameter(s["gq"]), torch.nn.Parameter(s["f"])
    side = [t for t in (s["cache"].k, s["cache"].v, s["cache"].k_scale, s["cache"].v_scale)]
    start = [t.clone() for t in side]
    CALLS[name](s, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [s[r].clone() for r in RESULTS[name]] + [t.clone() for t in side]
    for t, u in zip(side, start):
        t.copy_(u)
    for r in RESULTS[name]:
        s[r].zero_()
    if name == "decode":
        s["qo"].copy_(s["q"])
    monkeypatch.setattr(beam, "_launch", None)             # the Python way would fail
    CALLS[name](s)
    torch.cuda.synchronize()
    for a, b in zip([s[r] for r in RESULTS[name]] + side, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


BAD = [
    ("rope", "q", lambda t: t[:, :5]), ("rope", "q", lambda t: t.float()), ("rope", "q", lambda t: t.half()),
    ("rope", "q", lambda t: t.cpu()), ("rope", "k", lambda t: t[:4]), ("rope", "k", lambda t: t.transpose(0, 1)),
    ("rope", "pos", lambda t: t.long()), ("rope", "pos", lambda t: t.cpu()), ("rope", "pos", lambda t: t[:3]),
    ("rope", "qo", lambda t: t.transpose(1, 2)), ("rope", "ko", lambda t: t[:, :1]), ("rope", "f", lambda t: None),
    ("rope", "f", lambda t: t.double()), ("rope", "f", lambda t: t[:8]), ("rope", "gq", lambda t: t[:32]),
    ("rope", "gk", lambda t: t.float()), ("rope", "qo", lambda t: t.expand(5, 6, 64)[:, ::2]),
    ("rope_cache", "v", lambda t: t[:, :1]), ("rope_cache", "slots", lambda t: t.long()),
    ("rope_cache", "slots", lambda t: t[::2]), ("write", "v", lambda t: t.float()), ("write", "slots", lambda t: t[1:]),
    ("read", "table", lambda t: t.long()), ("read", "table", lambda t: t.t()), ("read", "off", lambda t: t[1:]),
    ("read", "vr", lambda t: t[1:]), ("read", "first", lambda t: t[1:]), ("decode", "lens", lambda t: t[1:]),
    ("decode", "table", lambda t: t[1:]), ("decode", "table", lambda t: t.cpu()), ("decode", "out", lambda t: t.float()),
    ("decode", "lse", lambda t: t.double()), ("decode", "lse", lambda t: t[:, :3]), ("decode", "ws", lambda t: t.float()),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_bad_tensors_are_refused(i):
    name, key, spoil = BAD[i]
    s = binding_state()
    kept = {r: s[r].fill_(3.0).clone() for r in RESULTS[name] if r != key}
    s[key] = spoil(s[key])
    with pytest.raises((ValueError, TypeError)):
        CALLS[name](s)
    torch.cuda.synchronize()
    for r, t in kept.items():
        assert torch.equal(s[r], t)


def test_bad_cache_and_workspace_are_refused():
    s = binding_state()
    other = beam.kv_cache(beam.AttnCfg(6, 2, 64, 32, False, 0, 32), 4, beam.BEAM_FP8_E4M3)      # another page size
    for name in ("rope_cache", "write", "read", "decode"):
        with pytest.raises(ValueError):
            CALLS[name](dict(s, cache=other))
    f32 = beam.kv_cache(s["cfg"], 4, beam.BEAM_F32)
    with pytest.raises(beam.BeamError) as e:
        CALLS["decode"](dict(s, cache=f32))
    assert e.value.status == 2                              # bf16 queries over an fp32 cache
    c = beam.AttnCfg(6, 2, 64, 0, False, 0, 16)
    table = torch.zeros((1, 200), dtype=torch.int32, device=DEV)
    with pytest.raises(beam.BeamError) as e:
        beam.beam_moe_attn_decode(c, s["qo"][:1], s["cache"], table, s["lens"][:1], 3000, s["out"][:1], s["ws"])
    assert e.value.status == 3                              # many parts, little workspace


def test_configurations_and_caches_copy():
    """Copies have handles of their own."""
    import copy
    import pickle
    s = binding_state()
    CALLS["decode"](s)
    want = s["out"].clone()
    for cfg in (copy.copy(s["cfg"]), copy.deepcopy(s["cfg"]), pickle.loads(pickle.dumps(s["cfg"]))):
        s["out"].zero_()
        CALLS["decode"](dict(s, cfg=cfg))
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want)
    c = s["cache"]
    again = beam.KVCache(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone())
    CALLS["decode"](dict(s, cache=again))
    torch.cuda.synchronize()
    assert torch.equal(s["out"], want)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_padded_batch(kind):
    """Idle rows of a step (slot -1, length 0, no pages, NaN inputs, any
    position) get a zero result, store nothing and change no other row."""
    cfg, table, c, qkv, gq, gk, f, pos, slots = step_state(kind, seed=5)
    B = qkv.shape[1]
    bufs = beam.attn_buffers(cfg, B, 1024, keep_lse=True)
    sides = [x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]
    before = [x.clone() for x in sides]
    beam.attn_layer(cfg, qkv[0], pos[0], slots[0], c, torch.tensor(table, device=DEV), pos[0] + 1, 1024, bufs, f, gq, gk)
    torch.cuda.synchronize()
    want, after = (bufs.out.clone(), bufs.lse.clone()), [x.clone() for x in sides]
    for x, y in zip(sides, before):
        x.copy_(y)
    # the same rows with idle ones between them
    at = [0, 2, 3, 5, 8, 10]
    N = 12
    spread = lambda x, fill: torch.full((N,) + tuple(x.shape[1:]), fill, dtype=x.dtype, device=DEV)
    q, p, s, n, t = (spread(qkv[0], float("nan")), spread(pos[0], -1), spread(slots[0], -1), spread(pos[0], 0),
                     spread(torch.tensor(table, device=DEV), -1))
    q[at], p[at], s[at], n[at], t[at] = qkv[0], pos[0], slots[0], pos[0] + 1, torch.tensor(table, device=DEV)
    big = beam.attn_buffers(cfg, N, 1024, keep_lse=True)
    beam.attn_layer(cfg, q, p, s, c, t, n, 1024, big, f, gq, gk)
    torch.cuda.synchronize()
    idle = [i for i in range(N) if i not in at]
    assert (big.out[idle] == 0).all() and torch.isneginf(big.lse[idle]).all()
    # the same split of each sequence, so the same bits
    assert torch.equal(big.out[at], want[0]) and torch.equal(big.lse[at], want[1])
    for x, y in zip(sides, after):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
