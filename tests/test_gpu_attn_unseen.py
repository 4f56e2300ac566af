"""GPU tests of what attention does not see: NaN there changes no bit of any
result, in decode and for new tokens, and outputs that are not numbers count as
wrong.

Tolerances of decode are those of test_gpu_attn_prompt.py's head: a score is off
by e = (D / 4 + 8) u Z, which moves a probability by the factor 1 + 2 e; sums of
n terms add c = (n / 32 + 64) u; over bf16, e4m3 and 4-bit caches a probability
is two bf16 parts, 2^-15 off (and 2 u with the value's scale); the result is
rounded once, by half a step, which below the least normal number is 2^-134.
"""

import numpy as np
import pytest
import torch

import oracle
import test_gpu_attn as base
import test_gpu_attn_prompt as prompts
from parity_util import over_bound, say

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
KINDS = prompts.KINDS
f64, gen, i32, filled, act_of = base.f64, base.gen, prompts.i32, prompts.filled, prompts.act_of


def decode_ref(cfg, kind, q, vals, table, lens, n_pages):
    """(out, bound, lse, bound) of one token per sequence."""
    B, hq, D = q.shape
    hkv = cfg.n_kv_heads
    out, eo, lse, el = np.zeros((B, hq, D)), np.zeros((B, hq, D)), np.zeros((B, hq)), np.zeros((B, hq))
    for b, L in enumerate(lens):
        L = min(max(L, 0), np.asarray(table).shape[1] * cfg.page_size)
        toks = np.nonzero(oracle.seen(1, L, cfg.window, cfg.sinks)[0])[0] if L else []
        kr, there = oracle.cached_rows(vals[0], table[b], toks, n_pages)
        vr, _ = oracle.cached_rows(vals[1], table[b], toks, n_pages)
        kr, vr = kr[there], vr[there]
        qb = f64(q[b]).reshape(hkv, hq // hkv, D)
        o, z, mag = (x.reshape(hq, -1) for x in oracle.decode_attention(qb, kr, vr, cfg.softmax_scale))
        Z = cfg.softmax_scale * max((np.abs(qb[h]) @ np.abs(kr[:, h]).T).max() for h in range(hkv)) if len(kr) else 0.0
        e, c = (D / 4 + 8) * U * Z, (len(kr) / 32 + 64) * U
        p_err = 0.0 if kind == "f32" else 2.0 ** -15 + 2 * U
        out[b], lse[b] = o, z[:, 0]
        eo[b] = (p_err + 2 * e + c) * mag + prompts.HALF[q.dtype] * np.abs(o) + 2.0 ** -134
        el[b] = e + c + U * np.abs(np.where(np.isinf(lse[b]), 0, lse[b]))
    return out, eo, lse, el


def run_decode(cfg, q, c, table, lens, max_len):
    B, hq, _ = q.shape
    out, lse = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV), torch.full((B, hq), 9.0, device=DEV)
    ws = beam.attn_workspace(cfg, B, max_len)
    ws.fill_(0xFF)                                          # its contents do not matter
    beam.beam_moe_attn_decode(cfg, q, c, i32(table), i32(lens), max_len, out, ws, lse)
    torch.cuda.synchronize()
    return out, lse


def check_decode(cfg, kind, q, c, vals, table, lens, max_len, name):
    out, lse = run_decode(cfg, q, c, table, lens, max_len)
    ro, eo, rl, el = decode_ref(cfg, kind, q, vals, table, lens, c.k.shape[0])
    got, gl, none = f64(out), f64(lse), np.isneginf(rl)
    over, lover = over_bound(got, ro, eo), over_bound(gl[~none], rl[~none], el[~none])
    say(f"  {name}: out over the bound by {over:.2e}, lse by {lover:.2e}")
    assert over <= 0 and lover <= 0, name
    assert np.array_equal(np.isneginf(gl), none) and (got[none] == 0).all()
    return out, lse


def poison(cfg, kind, c, seen):
    """NaN in every place of the cache c where seen [n_pages, P] is false."""
    bad = prompts.poisoned(cfg, c.k.shape[0], kind)
    keep = torch.tensor(seen, device=DEV)[:, None, :]
    for t, p in ((c.k, bad.k), (c.v, bad.v), (c.k_scale, bad.k_scale), (c.v_scale, bad.v_scale)):
        if t is not None:
            a, z = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (t, p))
            a.copy_(torch.where(keep if a.dim() == 3 else keep[..., None], a, z))


def places_seen(table, new, lens, P, n_pages, window, sinks):
    seen = np.zeros((n_pages, P), bool)
    for b, L in enumerate(lens):
        for j in np.nonzero(oracle.seen(new[b], L, window, sinks).any(0))[0]:
            seen[table[b, j // P], j % P] = True
    return seen


def same(a, b):
    return all(torch.isfinite(x).all() and torch.equal(x, y) for x, y in zip(a, b))


SHAPES = [(48, 8, 128), (4, 4, 64), (40, 1, 128), (48, 1, 64), (16, 1, 256), (40, 2, 256)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,D", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (33, 0), (33, 5), (64, 16), (500, 100)])
def test_decode_unseen_places_change_nothing(kind, hq, hkv, D, window, sinks):
    say(f"decode unseen {kind} {hq}/{hkv} D={D} window={window} sinks={sinks}")
    P, lens = 16, [1, 16, 47, 64, 65, 515, 640, 700]
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    n_pages = sum(-(-x // P) for x in lens) + 4
    c, vals = filled(cfg, n_pages, kind, 77)
    table = base.tables(lens, P, n_pages, 78)
    q = torch.randn((len(lens), hq, D), generator=gen(79), device=DEV).to(act_of(kind))
    clean = check_decode(cfg, kind, q, c, vals, table, lens, 700, "clean")
    poison(cfg, kind, c, places_seen(table, [1] * len(lens), lens, P, n_pages, window, sinks))
    assert same(run_decode(cfg, q, c, table, lens, 700), clean)
    assert same(run_decode(cfg, q, c, table, lens, 700), clean)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,hkv,lens,max_len,window,sinks", [
    (3, 2, [5000, 1, 4100], 5000, 0, 0), (3, 2, [5000, 1, 4100], 5000, 3000, 700), (1, 1, [9000], 9000, 8000, 33),
    (5, 2, [1700, 30, 1, 900, 7], 100, 600, 600), (40, 64, [3000] + [20] * 39, 70000, 2500, 300),
    (40, 64, [3000] + [20] * 39, 70000, 0, 0), (64, 8, [1000, 30, 999] + [500] * 61, 1000, 512, 100000),
])
def test_decode_in_parts(kind, B, hkv, lens, max_len, window, sinks):
    """Sequences in parts, joined and listed, and with sinks that reach every token; NaN behind the lengths."""
    say(f"decode parts {kind} B={B} window={window} sinks={sinks}")
    cfg = beam.AttnCfg(hkv, hkv, 64, 0, False, window, 64, softmax_scale=0.125, sinks=sinks)
    n_pages = sum(-(-n // 64) for n in lens) + 2
    c, vals = filled(cfg, n_pages, kind, 71)
    table = base.tables(lens, 64, n_pages, 72)
    q = torch.randn((B, hkv, 64), generator=gen(73), device=DEV).to(act_of(kind))
    clean = check_decode(cfg, kind, q, c, vals, table, lens, max_len, "parts")
    poison(cfg, kind, c, places_seen(table, [1] * B, lens, 64, n_pages, window, sinks))
    assert same(run_decode(cfg, q, c, table, lens, max_len), clean)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 0), (33, 5), (500, 100)])
def test_decode_bad_pages(kind, window, sinks):
    """Pages outside the cache are skipped; lengths below zero and beyond the table."""
    P, n_pages = 16, 40
    cfg = beam.AttnCfg(8, 2, 128, 0, False, window, P, sinks=sinks)
    lens, table = [100, 90, -5, 1 << 30], base.tables([100, 90, 1, 112], P, n_pages, 80, 7)
    table[0, 2], table[0, 5], table[1, :] = -1, n_pages, 1 << 20
    c, vals = filled(cfg, n_pages, kind, 81)
    q = torch.randn((4, 8, 128), generator=gen(79), device=DEV).to(act_of(kind))
    check_decode(cfg, kind, q, c, vals, table, lens, 112, "bad pages")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,D", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 0), (48, 5), (1, 1)])
def test_prompts_unseen_places_change_nothing(kind, hq, hkv, D, window, sinks):
    say(f"prompt unseen {kind} {hq}/{hkv} D={D} window={window} sinks={sinks}")
    P, new, lens = 16, [3, 1, 90, 10, 2], [70, 33, 130, 700, 2]
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    n_pages = sum(-(-x // P) for x in lens) + 4
    c, vals = filled(cfg, n_pages, kind, 17)
    table, off = prompts.sequences(new, lens, P, n_pages, 18)
    q = torch.randn((int(off[-1]), hq, D), generator=gen(19), device=DEV).to(act_of(kind))
    clean = prompts.run_prompt(cfg, q, c, table, off, lens, 700)
    ro, rl, eo, el = prompts.prompt_ref(cfg, kind, q, *vals, table, off, lens, n_pages)
    assert over_bound(f64(clean[0]), ro, eo) <= 0 and over_bound(f64(clean[1]), rl, el) <= 0
    poison(cfg, kind, c, places_seen(table, new, lens, P, n_pages, window, sinks))
    assert same(prompts.run_prompt(cfg, q, c, table, off, lens, 700), clean)
    assert same(prompts.run_prompt(cfg, q, c, table, off, lens, 700), clean)
