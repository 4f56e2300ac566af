"""GPU parity of the attention of new tokens (prompts, chunks, drafted and
single tokens), of sinks beside a window, and of the 4-bit key-value cache,
against the fp64 oracle (oracle/attn.py, oracle/moe.py).

Tolerances, from the arithmetic.  h(t) = finfo(t).eps / 2 is the relative
error of one rounding to t, u = h(fp32) = 2^-24.  With A = sum_j softmax_j |v_j|
and Z = scale * max_j sum_d |q_d k_jd|:

Prompts.  A score's products are exact (bf16, e4m3, 4 bits) or off by u each,
summed in at most D steps, and scaled in at most 3 roundings, so it is off by
e = (D + 8) u Z, which moves a probability by the factor 1 + 2 e; exp2, the
rescalings and the n-term sums in fp32 add c = (n / 32 + 64) u.  A probability
is rounded to bf16 once.  Over bf16 and 4-bit caches the sum is of the rounded
ones: with p_j (1 + d_j), |d_j| <= h(bf16), the result moves by
sum_j w_j d_j (v_j - out) / (1 + mean of d), at most
h(bf16) (A + |out|) (1 + 2 h(bf16)); over e4m3 caches p_j times the value's scale
(2 u) is rounded and the sum is not, which leaves h(bf16) A.  So out is off by
that + (2 e + c) A + h(dtype) |out|, and lse, whose sum is of the probabilities
as they were, by e + c + u |lse|.

Decode: the bound of tests/test_gpu_attn.py, with a probability as two bf16
parts (2^-15 off).  Below the least normal number a rounding is not off by a
share of the value but by half the step there, which adds 2^-134 (bf16, least step
2^-133) to a result's bound.

4-bit codes: an element's scaling is by a power of two and its rounding the
definition's, so codes and scales of given rows are equal, byte for byte; of
rows that were normed and rotated first (each element off by at most
2^-18 M + nothing, M the row's largest magnitude, stored from fp32), the value
is within half a step of the block's grid (which, for a block of exponent E, is
at most 2^(E+1) above 4 and 2 above the largest value 6: a value in [6, 8) times
2^E is stored as 6) of the exact one, plus that error; where the exact
largest magnitude lies within that error of a power of two, either scale may
be taken.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import synth
import test_gpu_attn as base
from parity_util import say

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = base.HALF
f64, gen = base.f64, base.gen
KINDS = ["bf16", "fp8", "fp4", "f32"]
CODE = dict(base.KIND, fp4=beam.BEAM_MXFP4)


def act_of(kind):
    return torch.float32 if kind == "f32" else torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def mx_values(codes, scale):
    """fp64 values of 4-bit rows."""
    c = codes.cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    return oracle.e2m1_decode(c) * np.repeat(oracle.e8m0_decode(scale.cpu().numpy()), 32, -1)


def filled(cfg, n_pages, kind, seed):
    """A cache of random rows, and its exact values k, v [n_pages, h, P, D]."""
    if kind != "fp4":
        return base.filled(cfg, n_pages, kind, seed)
    c = beam.kv_cache(cfg, n_pages, beam.BEAM_MXFP4, DEV)
    g = gen(seed)
    vals = []
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV))
        s.copy_(torch.randint(123, 128, s.shape, generator=g, device=DEV))
        vals.append(mx_values(t, s))
    return c, vals


def poisoned(cfg, n_pages, kind):
    """A cache whose every element is NaN."""
    if kind != "fp4":
        return base.poisoned(cfg, n_pages, kind)
    c = beam.kv_cache(cfg, n_pages, beam.BEAM_MXFP4, DEV)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.fill_(0xFF)
    return c


def sequences(new, lens, P, n_pages, seed, width=None):
    table = base.tables([max(n, 1) for n in lens], P, n_pages, seed, width)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return table, off


def prompt_ref(cfg, kind, q, k, v, table, off, lens, n_pages):
    """(out, lse, bound on out, bound on lse) of the rows below off[-1]."""
    T, hq, D = int(off[-1]), cfg.n_heads, cfg.head_dim
    hkv = cfg.n_kv_heads
    G, act = hq // hkv, q.dtype
    out, eo = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse, el = np.zeros((T, hq)), np.zeros((T, hq))
    for b, n in enumerate(np.diff(off)):
        if n == 0:
            continue
        L = min(max(lens[b], 0), table.shape[1] * cfg.page_size)
        kr, there = oracle.cached_rows(k, table[b], range(L), n_pages)
        vr, _ = oracle.cached_rows(v, table[b], range(L), n_pages)
        mask = oracle.seen(n, L, cfg.window, cfg.sinks) & there[None, :]
        use = mask.any(0)
        kr, vr, mask = kr[use], vr[use], mask[:, use]
        at = slice(off[b], off[b + 1])
        qb = f64(q[at]).reshape(n, hkv, G, D)
        o, z, mag = oracle.masked_attention(qb, kr, vr, mask, cfg.softmax_scale)
        Z = 0.0
        if len(kr):
            Z = cfg.softmax_scale * max(float((np.abs(qb[:, h].reshape(-1, D)) @ np.abs(kr[:, h]).T).max())
                                        for h in range(hkv))
        e, c = (D + 8) * U * Z, (len(kr) / 32 + 64) * U
        o, mag, z = o.reshape(n, hq, D), mag.reshape(n, hq, D), z.reshape(n, hq)
        hp = HALF[torch.bfloat16]
        p_err = 0.0 if kind == "f32" else (hp + 2 * U) * mag if kind == "fp8" else hp * (1 + 2 * hp) * (mag + np.abs(o))
        out[at], lse[at] = o, z
        eo[at] = p_err + (2 * e + c) * mag + HALF[act] * np.abs(o)
        el[at] = e + c + U * np.abs(np.where(np.isinf(z), 0, z))
    return out, lse, eo, el


def run_prompt(cfg, q, c, table, off, lens, max_len, lse=True, stream=None):
    T, B = q.shape[0], len(lens)
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    ls = torch.full((T, cfg.n_heads), 9.0, device=DEV) if lse else None
    ws = beam.attn_prompt_workspace(cfg, B, T, max_len)
    ws.fill_(0xFF)                                          # its contents do not matter
    beam.beam_moe_attn_prompt(cfg, q, c, i32(table), i32(off), i32(lens), max_len, out, ws, ls, stream)
    torch.cuda.synchronize()
    return out, ls


def check_prompt(cfg, kind, q, c, vals, table, off, lens, max_len, name, lse=True, n_pages=None):
    out, ls = run_prompt(cfg, q, c, table, off, lens, max_len, lse)
    ro, rl, eo, el = prompt_ref(cfg, kind, q, *vals, np.asarray(table), off, lens, n_pages or c.k.shape[0])
    T = int(off[-1])
    got = f64(out)
    assert (got[T:] == 9).all(), "rows behind the last sequence"
    d = np.abs(got[:T] - ro) - eo
    inf = np.isinf(rl)
    say(f"  {name}: out over the bound by {d.max():.2e}, rel {np.linalg.norm(got[:T] - ro) / max(np.linalg.norm(ro), 1e-30):.2e}")
    assert (d <= 0).all(), name
    assert (got[:T][np.broadcast_to(inf[..., None], ro.shape)] == 0).all()
    if lse:
        gl = f64(ls)
        assert (gl[T:] == 9).all()
        gl = gl[:T]
        assert np.array_equal(np.isneginf(gl), inf), name
        worst = np.max(np.abs(gl[~inf] - rl[~inf]) - el[~inf], initial=-1)
        say(f"  {name}: lse over the bound by {worst:.2e}")
        assert worst <= 0, name
    return out, ls


NEW = [0, 0, 1, 1, 5, 7, 130, 64, 33, 9, 1]
LEN = [0, 17, 1, 300, 5, 40, 130, 100, 513, 4, 64]     # the last but one: more new tokens than the sequence has


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,D", [(48, 8, 128), (4, 4, 64), (16, 1, 256), (17, 1, 128), (48, 1, 64), (64, 1, 128),
                                      (40, 2, 256), (6, 2, 64)])
@pytest.mark.parametrize("window,sinks,P", [(0, 0, 16), (100, 0, 64), (40, 4, 16), (33, 37, 32)])
def test_prompt(kind, hq, hkv, D, window, sinks, P):
    say(f"prompt {kind} {hq}/{hkv} D={D} window={window} sinks={sinks} P={P}")
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    n_pages = sum(-(-max(n, 1) // P) for n in LEN) + 2
    c, vals = filled(cfg, n_pages, kind, 7)
    table, off = sequences(NEW, LEN, P, n_pages, 1)
    T = int(off[-1]) + 3
    q = (torch.randn((T, hq, D), generator=gen(2), device=DEV) * 2).to(act_of(kind))
    check_prompt(cfg, kind, q, c, vals, table, off, LEN, max(LEN), "prompt")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,n,L", [(48, 8, 1, 5000), (48, 8, 16, 3001), (8, 1, 40, 2000), (16, 2, 3, 300),
                                        (64, 1, 5, 4100)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 9)])
def test_few_rows_over_a_long_cache(kind, hq, hkv, n, L, window, sinks):
    """Blocks cut into parts, and joined; a length that was not expected, too."""
    say(f"split prompt {kind} {hq}/{hkv} n={n} L={L} window={window}")
    cfg = beam.AttnCfg(hq, hkv, 128, 0, False, window, 64, sinks=sinks)
    new, lens = [n, 1], [L, L // 3]
    n_pages = sum(-(-x // 64) for x in lens) + 1
    c, vals = filled(cfg, n_pages, kind, 3)
    table, off = sequences(new, lens, 64, n_pages, 4)
    q = torch.randn((n + 1, hq, 128), generator=gen(5), device=DEV).to(act_of(kind))
    for max_len in (L, 100, 4 * L):
        check_prompt(cfg, kind, q, c, vals, table, off, lens, max_len, f"expected {max_len}", lse=max_len != 100)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 20)])
def test_single_tokens_beside_chunks(kind, window, sinks):
    """Many blocks, of which only the sequences in one are cut into parts."""
    say(f"mixed {kind} window={window}")
    cfg = beam.AttnCfg(16, 8, 64, 0, False, window, 32, softmax_scale=0.125, sinks=sinks)
    new, lens = [1, 1, 700, 0, 3, 2, 1, 4096 // 2], [3000, 1, 900, 50, 2500, 1100, 1030, 2048]
    n_pages = sum(-(-x // 32) for x in lens) + 1
    c, vals = filled(cfg, n_pages, kind, 13)
    table, off = sequences(new, lens, 32, n_pages, 14)
    q = torch.randn((int(off[-1]), 16, 64), generator=gen(15), device=DEV).to(act_of(kind))
    check_prompt(cfg, kind, q, c, vals, table, off, lens, 3000, "mixed")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 0), (48, 5), (16, 16), (1, 0), (1, 1)])
def test_prompt_garbage_where_no_row_sees(kind, window, sinks):
    """NaN behind the length, before the windows and in free pages."""
    say(f"prompt garbage {kind} window={window} sinks={sinks}")
    P = 16
    cfg = beam.AttnCfg(12, 2, 128, 0, False, window, P, sinks=sinks)
    new, lens = [3, 1, 30, 10], [70, 33, 130, 200]
    n_pages = sum(-(-x // P) for x in lens) + 4
    c, vals = filled(cfg, n_pages, kind, 17)
    table, off = sequences(new, lens, P, n_pages, 18)
    seen = np.zeros((n_pages, P), bool)
    for b, L in enumerate(lens):
        for j in np.nonzero(oracle.seen(new[b], L, window, sinks).any(0))[0]:
            seen[table[b, j // P], j % P] = True
    bad = poisoned(cfg, n_pages, kind)
    keep = torch.tensor(seen, device=DEV)[:, None, :]
    for t, p in ((c.k, bad.k), (c.v, bad.v), (c.k_scale, bad.k_scale), (c.v_scale, bad.v_scale)):
        if t is not None:
            a, z = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (t, p))
            a.copy_(torch.where(keep if a.dim() == 3 else keep[..., None], a, z))
    q = torch.randn((int(off[-1]), 12, 128), generator=gen(19), device=DEV).to(act_of(kind))
    check_prompt(cfg, kind, q, c, vals, table, off, lens, 200, "garbage")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,D", [(12, 2, 128), (4, 4, 64), (6, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_values_that_are_not_finite_reach_who_sees_them(kind, hq, hkv, D, window, sinks):
    """NaN keys, NaN and infinite values at some tokens: rows that do not see
    those are the same bits as without, rows that do are NaN."""
    say(f"prompt not finite {kind} {hq}/{hkv} D={D}")
    P, n, L = 16, 90, 150
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    c, vals = filled(cfg, 12, kind, 21)
    table, off = sequences([n], [L], P, 12, 22)
    q = torch.randn((n, hq, D), generator=gen(23), device=DEV).to(act_of(kind))
    clean, _ = run_prompt(cfg, q, c, table, off, [L], L)
    for bad in ([70], [149], [61, 100], [1], [95]):
        w, _ = filled(cfg, 12, kind, 21)
        for i, t in enumerate(bad):
            pg, at = table[0, t // P], t % P
            if kind == "fp4":
                w.v_scale[pg, 0, at, -1] = 255
            elif kind == "fp8" and i == 0:
                w.v.view(torch.uint8)[pg, 0, at, D // 2] = 0x7F
            elif kind == "fp8":
                w.v_scale[pg, 0, at] = float("inf")
            else:
                w.v[pg, 0, at, D - 1] = float("inf" if i else "nan")
            if t == 95:
                (w.k_scale[pg, 0, at].fill_(255) if kind == "fp4" else
                 w.k.view(torch.uint8)[pg, 0, at].fill_(0x7F) if kind == "fp8" else w.k[pg, 0, at].fill_(float("nan")))
        got, _ = run_prompt(cfg, q, w, table, off, [L], L)
        mask = oracle.seen(n, L, window, sinks)
        sees = mask[:, bad].any(1)
        G = hq // hkv
        a, b = f64(got), f64(clean)
        assert np.array_equal(a[:, G:], b[:, G:])            # the other heads
        assert np.array_equal(a[~sees], b[~sees]), bad
        assert (~np.isfinite(a[sees][:, :G])).any(-1).all(), bad
        if kind in ("bf16", "f32") and bad != [95]:          # only the element that is not finite
            assert np.array_equal(a[sees][:, :G, :D - 1], b[sees][:, :G, :D - 1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(12, 2, 128), (4, 4, 64), (6, 1, 256)])
@pytest.mark.parametrize("n,L", [(1, 20), (1, 150), (7, 100), (90, 150), (1, 3000), (200, 200)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (7, 0)])
def test_infinite_values_stay_infinite(kind, hq, hkv, D, n, L, window, sinks):
    """A weight above 0 times an infinite value: also where it is the first
    token that a row sees, and in one of the halves that pairs of waves take.
    Scores differ by far less than what makes a weight 0."""
    P = 16
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    pages = -(-L // P) + 1
    c, _ = filled(cfg, pages, kind, 21)
    table, off = sequences([n], [L], P, pages, 22)
    q = torch.randn((n, hq, D), generator=gen(23), device=DEV).to(act_of(kind))
    clean, _ = run_prompt(cfg, q, c, table, off, [L], L)
    mask = oracle.seen(n, L, window, sinks)
    for t in sorted({0, L - 1, L - 2, L - 7, max(L - 40, 0), max(L - 41, 0), L // 2}):
        w, _ = filled(cfg, pages, kind, 21)
        w.v[table[0, t // P], 0, t % P, 5] = float("-inf" if t % 2 else "inf")
        got, lse = run_prompt(cfg, q, w, table, off, [L], L)
        want = f64(clean).copy()
        rows = np.nonzero(mask[:, t])[0]
        want[rows, :hq // hkv, 5] = -np.inf if t % 2 else np.inf
        assert np.array_equal(f64(got), want), t


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_bad_pages_and_lengths(kind):
    say(f"prompt bad pages {kind}")
    P = 16
    cfg = beam.AttnCfg(6, 2, 64, 0, False, 0, P, softmax_scale=0.125)
    lens, new = [100, 90, -5, 1 << 30, 64, 33], [40, 3, 2, 5, 64, 33]
    c, vals = filled(cfg, 40, kind, 25)
    table, off = sequences(new, [100, 90, 1, 112, 64, 33], P, 40, 26, width=7)
    table[0, 2], table[0, 5], table[1, :] = -1, 40, 1 << 20
    table[4, 0], table[4, 3] = -(1 << 31), (1 << 31) - 1
    q = torch.randn((int(off[-1]), 6, 64), generator=gen(27), device=DEV).to(act_of(kind))
    check_prompt(cfg, kind, q, c, vals, table, off, lens, 112, "bad pages")
    # no table at all
    out, ls = run_prompt(cfg, q, c, np.zeros((6, 0), np.int32), off, lens, 112)
    assert (f64(out) == 0).all() and np.isneginf(f64(ls)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_that_do_not_ascend_touch_nothing_else(kind):
    """Offsets below 0, beyond T or going back: only rows 0 .. T - 1 are written."""
    cfg = beam.AttnCfg(6, 2, 64, 0, False, 0, 16, softmax_scale=0.125)
    c, _ = filled(cfg, 10, kind, 25)
    table, _ = sequences([1, 1, 1], [40, 40, 40], 16, 10, 26)
    big = torch.full((30, 6, 64), 9.0, dtype=act_of(kind), device=DEV)
    q = torch.randn((10, 6, 64), generator=gen(27), device=DEV).to(act_of(kind))
    for off in ([0, 20, 5, 10], [-7, 3, 1 << 30, 2], [10, 8, 4, 0], [5, 5, 5, 5], [0, 10, 10, 10]):
        ws = beam.attn_prompt_workspace(cfg, 3, 10, 40)
        beam.beam_moe_attn_prompt(cfg, q, c, i32(table), i32(off), i32([40, 40, 40]), 40, big[10:20], ws)
        torch.cuda.synchronize()
        assert (big[:10] == 9).all() and (big[20:] == 9).all(), off


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_scores_far_apart(kind):
    """Scores hundreds apart in ascending and descending order, alternating, and
    constant: the running reference moves in every way."""
    say(f"prompt scores {kind}")
    P, L, n, D = 16, 400, 300, 64
    cfg = beam.AttnCfg(2, 1, D, 0, False, 0, P, softmax_scale=1.0)
    c, vals = filled(cfg, 26, kind, 31)
    table, off = sequences([n], [L], P, 26, 32)
    q = torch.zeros((n, 2, D), device=DEV)
    q[:, 0, 0], q[:, 1, 0] = 8.0, -8.0
    for order in ("up", "down", "alternating", "same"):
        t = np.arange(L)
        x = {"up": t, "down": L - t, "alternating": np.where(t % 3 == 0, t, -t), "same": np.full(L, 200)}[order] // 4 / 4.0
        row = np.zeros((L, D), np.float32)
        row[:, 0] = x
        k = torch.tensor(row, device=DEV)[:, None]
        slots = i32([int(table[0, i // P]) * P + i % P for i in range(L)])
        v = torch.randn((L, 1, D), generator=gen(33), device=DEV)
        beam.beam_moe_kv_write(cfg, k, v, slots, c)
        ko, vo = (torch.empty((26 * P, 1, D), device=DEV) for _ in range(2))
        every = torch.arange(26, dtype=torch.int32, device=DEV)[None]
        beam.beam_moe_kv_read(cfg, c, every, i32([0, 26 * P]), ko, vo)
        vals = [f64(y).reshape(26, P, 1, D).transpose(0, 2, 1, 3) for y in (ko, vo)]
        check_prompt(cfg, kind, q.to(act_of(kind)), c, vals, table, off, [L], L, order)


@pytest.mark.parametrize("kind", ["bf16", "fp4", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (16, 1, 64), (6, 2, 256)])
def test_equal_values_come_back(kind, hq, hkv, D):
    """The weights sum to one as they enter the product: a row whose values are all the same gets them back,
    but for the accumulation's fp32 roundings and one to the output."""
    P, L, n = 16, 500, 120
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 0, P, softmax_scale=D ** -0.5)
    c, _ = filled(cfg, 32, kind, 35)
    table, off = sequences([n], [L], P, 32, 36)
    row = torch.randint(-3, 4, (hkv, D), generator=gen(37), device=DEV).float()      # on every grid (4 bits: 1 .. 3)
    k = torch.randn((L, hkv, D), generator=gen(38), device=DEV)
    slots = i32([int(table[0, i // P]) * P + i % P for i in range(L)])
    row[:, ::32] = 3.0                                         # a block's largest magnitude
    beam.beam_moe_kv_write(cfg, k, row.expand(L, hkv, D).contiguous(), slots, c)
    q = torch.randn((n, hq, D), generator=gen(39), device=DEV).to(act_of(kind)) * 3
    out, _ = run_prompt(cfg, q, c, table, off, [L], L)
    want = f64(row).repeat(hq // hkv, 0)[None]
    # bf16 holds these integers: what is off by less than half a step comes back as it is
    assert np.abs(f64(out) - want).max() <= (0 if kind != "f32" else 3 * (L / 32 + 64) * U)


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_in_chunks_and_one_by_one(kind):
    """A prompt in one call, in chunks and token by token (through decode, too)."""
    say(f"chunks {kind}")
    P, L, hq, hkv, D = 32, 210, 12, 2, 128
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 64, P, sinks=3)
    c, vals = filled(cfg, 8, kind, 41)
    table, off = sequences([L], [L], P, 8, 42)
    q = torch.randn((L, hq, D), generator=gen(43), device=DEV).to(act_of(kind))
    whole, lse = check_prompt(cfg, kind, q, c, vals, table, off, [L], L, "whole")
    ro, _, eo, _ = prompt_ref(cfg, kind, q, *vals, table, off, [L], 8)
    for size in (1, 37, 64):
        for i in range(0, L, size):
            m = min(size, L - i)
            part, _ = run_prompt(cfg, q[i:i + m], c, table, [0, m], [i + m], L)
            assert (np.abs(f64(part) - ro[i:i + m]) <= eo[i:i + m]).all(), (size, i)
    out = torch.empty((L, hq, D), dtype=q.dtype, device=DEV)
    beam.beam_moe_attn_decode(cfg, q, c, i32(np.repeat(table, L, 0)), i32(range(1, L + 1)), L, out,
                              beam.attn_workspace(cfg, L, L))
    assert (np.abs(f64(out) - ro) <= eo).all()


def test_prompt_many_sequences_strided_queries():
    P, B, hq, hkv, D = 16, 3000, 6, 2, 64
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 20, P, softmax_scale=0.125, sinks=2)
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, B).tolist()
    new = [int(rng.integers(0, 4)) if x == 0 else int(min(x, rng.integers(0, 12))) for x in lens]
    n_pages = sum(-(-max(x, 1) // P) for x in lens) + 1
    c, vals = filled(cfg, n_pages, "bf16", 44)
    table, off = sequences(new, lens, P, n_pages, 45, 3)
    T = int(off[-1])
    wide = torch.randn((T, hq * D + 3 * D), generator=gen(46), device=DEV).to(torch.bfloat16)
    q = wide[:, D:D + hq * D].unflatten(1, (hq, D))
    check_prompt(cfg, "bf16", q, c, vals, table, off, lens, 40, "many")


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_prompt_over_cache_offsets_beyond_32_bits(kind):
    """Pages at the far end of a cache of more than 2^32 bytes (bf16) or elements."""
    hkv, D, P = 8, 256, 1024
    n_pages = (1 << 33) // (hkv * D * P) // (1 if kind == "fp4" else 2) + 3
    cfg = beam.AttnCfg(8, hkv, D, 0, False, 0, P, softmax_scale=1 / 16)
    c = beam.kv_cache(cfg, n_pages, CODE[kind], DEV)
    table = np.array([[n_pages - 1, 0]], np.int32)
    k, v = (torch.randn((1100, hkv, D), generator=gen(47 + i), device=DEV) for i in range(2))
    slots = i32([int(table[0, i // P]) * P + i % P for i in range(1100)])
    beam.beam_moe_kv_write(cfg, k, v, slots, c)
    ko, vo = (torch.empty_like(k) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, i32(table), i32([0, 1100]), ko, vo)
    want = [oracle.quantize_mx_fp4(f64(x).reshape(-1, D)) for x in (k, v)] if kind == "fp4" else None
    if kind == "fp4":
        for got, (s, e) in zip((ko, vo), want):
            assert np.array_equal(f64(got).reshape(-1, D), e * np.repeat(np.exp2(s.astype(float) - 127), 32, -1))
    else:
        assert torch.equal(ko, k.to(torch.bfloat16).float()) and torch.equal(vo, v.to(torch.bfloat16).float())
    vals = []
    for x in (ko, vo):
        p = np.zeros((2, hkv, P, D))
        p[0] = f64(x)[:P].transpose(1, 0, 2)
        p[1, :, :76] = f64(x)[P:].transpose(1, 0, 2)
        vals.append(p)
    q = torch.randn((9, 8, D), generator=gen(49), device=DEV).to(torch.bfloat16)
    out, _ = run_prompt(cfg, q, c, table, [0, 9], [1100], 1100)
    ro, _, eo, _ = prompt_ref(cfg, kind, q, *vals, np.array([[0, 1]]), np.array([0, 9]), [1100], 2)
    assert (np.abs(f64(out) - ro) <= eo).all()
    del c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [4096, 1 << 30, (1 << 31) - 1])
def test_a_window_beyond_every_token_is_none(kind, window):
    """Also where a sequence has more new tokens than it is long, whose first
    queries stand before it: a query's position less such a window, counted in
    32 bits, would come out at their other end."""
    new, lens = [300, 1, 40, 0, 200], [300, 700, 1000, 5, 70]
    c0 = beam.AttnCfg(12, 2, 128, 0, False, 0, 16)
    n_pages = sum(-(-n // 16) for n in lens) + 2
    c, _ = filled(c0, n_pages, kind, 3)
    table, off = sequences(new, lens, 16, n_pages, 4)
    q = torch.randn((int(off[-1]), 12, 128), generator=gen(5), device=DEV).to(act_of(kind))
    want, wl = run_prompt(c0, q, c, table, off, lens, max(lens))
    for sinks in (0, 5, 1 << 30):
        cfg = beam.AttnCfg(12, 2, 128, 0, False, window, 16, sinks=sinks)
        got, gl = run_prompt(cfg, q, c, table, off, lens, max(lens))
        assert torch.equal(got, want) and torch.equal(gl, wl), sinks


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_prompt_in_a_graph_and_on_two_streams(kind):
    """Captured, replayed with other lengths, offsets and queries, with eager work between; two at once."""
    P, hq, hkv, D = 32, 12, 2, 128
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 300, P, sinks=4)
    c, vals = filled(cfg, 200, kind, 51)
    B, T, ml = 3, 40, 2000
    table, _ = sequences([1] * B, [ml] * B, P, 200, 52)
    t, q = i32(table), torch.randn((T, hq, D), generator=gen(53), device=DEV).to(torch.bfloat16)
    off, lens = i32([0, 1, 30, 40]), i32([500, 600, 2000])
    out, lse = torch.zeros_like(q), torch.zeros((T, hq), device=DEV)
    ws = beam.attn_prompt_workspace(cfg, B, T, ml)
    beam.beam_moe_attn_prompt(cfg, q, c, t, off, lens, ml, out, ws, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam.beam_moe_attn_prompt(cfg, q, c, t, off, lens, ml, out, ws, lse)
    for i, (o, n) in enumerate([([0, 1, 30, 40], [500, 600, 2000]), ([0, 0, 0, 3], [9, 0, 1999]),
                                ([0, 13, 26, 39], [13, 1300, 40]), ([0, 40, 40, 40], [2000, 1, 1])]):
        off.copy_(i32(o))
        lens.copy_(i32(n))
        q.copy_(torch.randn((T, hq, D), generator=gen(60 + i), device=DEV))
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        eager, el = run_prompt(cfg, q, c, table, o, n, ml)
        m = o[-1]
        assert torch.equal(out[:m], eager[:m]) and torch.equal(lse[:m], el[:m]) and (out[m:] == 9).all()
        ro, _, eo, _ = prompt_ref(cfg, kind, q, *vals, table, np.array(o), n, 200)
        assert (np.abs(f64(out[:m]) - ro) <= eo).all()
    # two calls at once, each with its workspace, on streams of their own
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    wss = [beam.attn_prompt_workspace(cfg, B, T, ml) for _ in range(2)]
    off.copy_(i32([0, 1, 30, 40]))
    lens.copy_(i32([500, 600, 2000]))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, wss):
            beam.beam_moe_attn_prompt(cfg, q, c, t, off, lens, ml, o, w, stream=s)
    torch.cuda.synchronize()
    eager, _ = run_prompt(cfg, q, c, table, [0, 1, 30, 40], [500, 600, 2000], ml, lse=False)
    assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)


# ------------------------------------------------------------------ decode: sinks and 4 bits

def check_decode(cfg, kind, q, c, vals, table, lens, max_len, name):
    """The bound of tests/test_gpu_attn.py, over the visible tokens."""
    B, D = len(lens), cfg.head_dim
    hkv, hq = cfg.n_kv_heads, cfg.n_heads
    out, lse = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV), torch.full((B, hq), 9.0, device=DEV)
    ws = beam.attn_workspace(cfg, B, max_len)
    ws.fill_(0xFF)
    beam.beam_moe_attn_decode(cfg, q, c, i32(table), i32(lens), max_len, out, ws, lse)
    torch.cuda.synchronize()
    got, gl, worst = f64(out), f64(lse), -1.0
    for b, L in enumerate(lens):
        L = min(max(L, 0), np.asarray(table).shape[1] * cfg.page_size)
        toks = np.nonzero(oracle.seen(1, L, cfg.window, cfg.sinks)[0])[0] if L else []
        kr, there = oracle.cached_rows(vals[0], table[b], toks, c.k.shape[0])
        vr, _ = oracle.cached_rows(vals[1], table[b], toks, c.k.shape[0])
        kr, vr = kr[there], vr[there]
        qb = f64(q[b]).reshape(hkv, hq // hkv, D)
        o, z, mag = oracle.decode_attention(qb, kr, vr, cfg.softmax_scale)
        Z = cfg.softmax_scale * max((np.abs(qb[h]) @ np.abs(kr[:, h]).T).max() for h in range(hkv)) if len(kr) else 0.0
        e, n = (D / 4 + 8) * U * Z, (len(kr) / 32 + 64) * U
        half_p = 0.0 if kind == "f32" else 2.0 ** -15 + 2 * U
        bound = (half_p + 2 * e + n) * mag.reshape(hq, D) + HALF[q.dtype] * np.abs(o.reshape(hq, D)) + 2.0 ** -134
        worst = max(worst, (np.abs(got[b] - o.reshape(hq, D)) - bound).max())
        z = z.reshape(hq)
        if not len(kr):
            assert (got[b] == 0).all() and np.isneginf(gl[b]).all()
        else:
            assert (np.abs(gl[b] - z) <= e + n + U * np.abs(z)).all(), (name, b)
    say(f"  {name}: out over the bound by {worst:.2e}")
    assert worst <= 0, name


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 300, 513]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,D", [(48, 8, 128), (4, 4, 64), (16, 1, 256), (17, 1, 128), (48, 1, 64), (64, 1, 128),
                                      (40, 2, 256), (6, 2, 64)])
@pytest.mark.parametrize("window,sinks,P", [(0, 0, 16), (100, 0, 64), (100, 4, 64), (33, 37, 16), (1, 1, 32),
                                            (16, 16, 16), (64, 1000, 64)])
def test_decode(kind, hq, hkv, D, window, sinks, P):
    if kind != "fp4" and sinks == 0:
        pytest.skip("in tests/test_gpu_attn.py")
    say(f"decode {kind} {hq}/{hkv} D={D} window={window} sinks={sinks} P={P}")
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5, sinks=sinks)
    n_pages = sum(-(-n // P) for n in LENS) + 2
    c, vals = filled(cfg, n_pages, kind, 7)
    table = base.tables(LENS, P, n_pages, 1)
    q = (torch.randn((len(LENS), hq, D), generator=gen(2), device=DEV) * 2).to(act_of(kind))
    check_decode(cfg, kind, q, c, vals, table, LENS, max(LENS), "decode")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,hkv,lens,max_len,window,sinks", [
    (3, 2, [5000, 1, 4100], 5000, 0, 0), (3, 2, [5000, 1, 4100], 5000, 3000, 700), (1, 1, [9000], 9000, 8000, 33),
    (5, 2, [1700, 30, 1, 900, 0], 100, 600, 600), (40, 64, [3000] + [20] * 39, 70000, 2500, 300),
])
def test_decode_parts(kind, B, hkv, lens, max_len, window, sinks):
    """Sequences in parts, joined; the last case lists its parts."""
    say(f"decode parts {kind} B={B} window={window} sinks={sinks}")
    cfg = beam.AttnCfg(hkv, hkv, 64, 0, False, window, 64, softmax_scale=0.125, sinks=sinks)
    n_pages = sum(-(-n // 64) for n in lens) + 2
    c, vals = filled(cfg, n_pages, kind, 71)
    table = base.tables(lens, 64, n_pages, 72)
    q = torch.randn((B, hkv, 64), generator=gen(73), device=DEV).to(act_of(kind))
    check_decode(cfg, kind, q, c, vals, table, lens, max_len, "parts")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (33, 5), (64, 16), (500, 100), (0, 0)])
def test_decode_garbage_where_it_does_not_see(kind, window, sinks):
    say(f"decode garbage {kind} window={window} sinks={sinks}")
    P, lens = 16, [1, 16, 47, 64, 65, 515, 640, 700]
    cfg = beam.AttnCfg(8, 2, 128, 0, False, window, P, sinks=sinks)
    n_pages = sum(-(-x // P) for x in lens) + 4
    c, vals = filled(cfg, n_pages, kind, 77)
    table = base.tables(lens, P, n_pages, 78)
    seen = np.zeros((n_pages, P), bool)
    for b, L in enumerate(lens):
        for j in np.nonzero(oracle.seen(1, L, window, sinks)[0])[0]:
            seen[table[b, j // P], j % P] = True
    bad = poisoned(cfg, n_pages, kind)
    keep = torch.tensor(seen, device=DEV)[:, None, :]
    for t, p in ((c.k, bad.k), (c.v, bad.v), (c.k_scale, bad.k_scale), (c.v_scale, bad.v_scale)):
        if t is not None:
            a, z = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (t, p))
            a.copy_(torch.where(keep if a.dim() == 3 else keep[..., None], a, z))
    q = torch.randn((len(lens), 8, 128), generator=gen(79), device=DEV).to(act_of(kind))
    check_decode(cfg, kind, q, c, vals, table, lens, 700, "garbage")
    lens2, t2 = [100, 90, -5, 1 << 30], base.tables([100, 90, 1, 112], P, n_pages, 80, 7)
    t2[0, 2], t2[0, 5], t2[1, :] = -1, n_pages, 1 << 20
    c, vals = filled(cfg, n_pages, kind, 81)
    check_decode(cfg, kind, q[:4], c, vals, t2, lens2, 112, "bad pages")


@pytest.mark.parametrize("hq,hkv,D", [(6, 1, 64), (48, 8, 128), (40, 1, 128), (4, 2, 256)])
def test_decode_of_uneven_queries_over_four_bits(hq, hkv, D):
    """Queries whose elements span many powers of two, huge and tiny ones, all zeros; and what is not finite."""
    P, L = 16, 70
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 0, P, softmax_scale=1.0)
    c, vals = filled(cfg, 6, "fp4", 95)
    table = base.tables([L] * 6, P, 30, 96, 5) % 6
    g = gen(97)
    q = torch.randn((6, hq, D), generator=g, device=DEV)
    q[0] *= torch.exp2(torch.randint(-30, 1, q[0].shape, generator=g, device=DEV).float())
    q[1] *= 2.0 ** -60
    q[2, :, ::32] = 100.0
    q[3] = 0
    q[4] *= torch.exp2(torch.randint(-140, -100, q[4].shape, generator=g, device=DEV).float())
    check_decode(cfg, "fp4", q.to(torch.bfloat16), c, vals, table, [L] * 6, L, "uneven queries")
    q[5, hq - 1, D - 1] = float("nan")
    out = torch.empty((6, hq, D), dtype=torch.bfloat16, device=DEV)
    beam.beam_moe_attn_decode(cfg, q.to(torch.bfloat16), c, i32(table), i32([L] * 6), L, out, beam.attn_workspace(cfg, 6, L))
    want = np.zeros((6, hq), bool)
    want[5, hq - 1] = True
    assert np.array_equal(torch.isnan(out).all(-1).cpu().numpy(), want)
    assert np.array_equal(torch.isnan(out).any(-1).cpu().numpy(), want)


def test_sinks_without_a_window_say_nothing():
    P, L = 16, 300
    a, b = (beam.AttnCfg(8, 2, 128, 0, False, 0, P, sinks=s) for s in (0, 40))
    c, _ = filled(a, 20, "bf16", 83)
    table = i32(base.tables([L], P, 20, 84))
    q = torch.randn((1, 8, 128), generator=gen(85), device=DEV).to(torch.bfloat16)
    outs = []
    for cfg in (a, b):
        o = torch.empty_like(q)
        beam.beam_moe_attn_decode(cfg, q, c, table, i32([L]), L, o, beam.attn_workspace(cfg, 1, L))
        p = torch.empty_like(q)
        beam.beam_moe_attn_prompt(cfg, q, c, table, i32([0, 1]), i32([L]), L, p, beam.attn_prompt_workspace(cfg, 1, 1, L))
        outs.append((o, p))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ------------------------------------------------------------------ the 4-bit cache

@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,hkv,D,P", [(1, 8, 128, 16), (5, 1, 64, 16), (131, 8, 128, 64), (70, 3, 256, 32),
                                       (1000, 2, 64, 128), (9, 256, 64, 16)])
def test_four_bit_rows(act, T, hkv, D, P):
    """Codes and scales byte for byte the definition's (and the layer's quantiser's), unwritten places as they
    were, rows read back exactly, in both types."""
    say(f"4-bit rows {act} T={T} {hkv} D={D}")
    cfg = beam.AttnCfg(hkv, hkv, D, 0, False, 0, P)
    n_pages = -(-T // P) + 2
    c = beam.kv_cache(cfg, n_pages, beam.BEAM_MXFP4, DEV)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.fill_(0xA5)
    g = gen(T + D)
    dt = base.ACT[act]
    m = torch.randn((T, 2 * hkv * D + 16), generator=g, device=DEV)
    m *= torch.exp2(torch.randint(-12, 12, (T, 1), generator=g, device=DEV).float())
    if T > 4:
        m[0] = 0.0
        m[1, ::3] = 0.0
        m[2] = torch.sign(m[2]) * 2.0 ** -130 if act == "f32" else 0.0
        m[3] = torch.round(m[3] * 4 / m[3].abs().max()) * 1.25     # ties
    m = m.to(dt)
    k, v = m[:, 8:8 + hkv * D].unflatten(1, (hkv, D)), m[:, 8 + hkv * D:8 + 2 * hkv * D].unflatten(1, (hkv, D))
    slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 2:
        slots[T // 2], slots[T - 1] = -1, n_pages * P
    beam.beam_moe_kv_write(cfg, k, v, slots, c)
    torch.cuda.synchronize()
    sl = slots.cpu().numpy()
    live = np.nonzero((sl >= 0) & (sl < n_pages * P))[0]
    for x, codes, scale in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        want_c, want_s = np.full(codes.shape, 0xA5, np.uint8), np.full(scale.shape, 0xA5, np.uint8)
        s, e = oracle.quantize_mx_fp4(f64(x)[live])
        # the oracle's element keeps no sign of zero; the code does
        q = oracle.e2m1_encode(np.copysign(np.abs(e), f64(x)[live]))
        want_c[sl[live] // P, :, sl[live] % P] = q[..., 0::2] | (q[..., 1::2] << 4)
        want_s[sl[live] // P, :, sl[live] % P] = s
        assert np.array_equal(scale.cpu().numpy(), want_s) and np.array_equal(codes.cpu().numpy(), want_c)
    # each token read back as a sequence of its own
    for out in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((T + 2, hkv, D), 9.0, dtype=out, device=DEV) for _ in range(2))
        ok = (slots >= 0) & (slots < n_pages * P)
        table = torch.where(ok, slots // P, -1)[:, None].to(torch.int32).contiguous()
        first = torch.where(ok, slots % P, 0).to(torch.int32)
        beam.beam_moe_kv_read(cfg, c, table, torch.arange(T + 1, dtype=torch.int32, device=DEV), ko, vo, first=first)
        torch.cuda.synchronize()
        for x, got in ((k, ko), (v, vo)):
            s, e = oracle.quantize_mx_fp4(f64(x))
            want = e * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, -1)
            dead = np.setdiff1d(np.arange(T), live)
            want[dead] = 0
            assert np.array_equal(f64(got)[:T], want) and (f64(got)[T:] == 9).all()


def test_four_bit_codes_are_the_layers_quantisers():
    """A head row's bytes are what beam_moe_quantize_mx gives the same elements."""
    cfg, T = beam.AttnCfg(8, 8, 128, 0, False, 0, 16), 64
    layer = beam.LayerCfg(hidden=1024)
    x = torch.randn((T, 1024), generator=gen(91), device=DEV).to(torch.bfloat16)
    xq, xs = torch.empty((T, 512), dtype=torch.uint8, device=DEV), torch.empty((T, 32), dtype=torch.uint8, device=DEV)
    beam.beam_moe_quantize_mx(layer, x, xq, xs)
    c = beam.kv_cache(cfg, 4, beam.BEAM_MXFP4, DEV)
    beam.beam_moe_kv_write(cfg, x.view(T, 8, 128), x.view(T, 8, 128), torch.arange(T, dtype=torch.int32, device=DEV), c)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert torch.equal(codes.transpose(1, 2).reshape(T, 512), xq)
        assert torch.equal(scale.transpose(1, 2).reshape(T, 32), xs)


def test_four_bit_rows_that_are_not_finite():
    """An infinite element reads back infinite, beside zeros; a NaN as 6 scales of the rest of its block."""
    cfg = beam.AttnCfg(1, 1, 64, 0, False, 0, 16)
    x = torch.ones((3, 1, 64), device=DEV)
    x[0, 0, 3], x[0, 0, 40] = float("inf"), float("-inf")
    x[1, 0, 5] = float("nan")
    x[2, 0, :32] = torch.finfo(torch.float32).max
    c = beam.kv_cache(cfg, 1, beam.BEAM_MXFP4, DEV)
    beam.beam_moe_kv_write(cfg, x, x, i32([0, 1, 2]), c)
    ko, vo = (torch.empty_like(x) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, i32([[0]]), i32([0, 3]), ko, vo)
    got = f64(ko)[:, 0]
    assert got[0, 3] == np.inf and got[0, 40] == -np.inf and (np.delete(got[0], [3, 40]) == 0).all()
    assert got[1, 5] == 1.5 and (np.delete(got[1], 5) == 1).all()
    assert (got[2, :32] == 6 * 2.0 ** 125).all() and (got[2, 32:] == 1).all()
    assert torch.equal(ko, vo)


def test_every_four_bit_code_and_scale_reads_back():
    cfg = beam.AttnCfg(1, 1, 64, 0, False, 0, 256)
    c = beam.kv_cache(cfg, 1, beam.BEAM_MXFP4, DEV)
    codes = torch.arange(64, device=DEV) % 16
    packed = (codes[0::2] | codes[1::2] << 4).to(torch.uint8)
    for t in (c.k, c.v):
        t.copy_(packed.expand_as(t))
    s = torch.arange(256, device=DEV)
    c.k_scale.copy_(torch.stack([s, s], -1).view(1, 1, 256, 2))
    c.v_scale.copy_(torch.stack([s, 255 - s], -1).view(1, 1, 256, 2))
    ko, vo = (torch.empty((256, 1, 64), device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, i32([[0]]), i32([0, 256]), ko, vo)
    for got, t, sc in ((ko, c.k, c.k_scale), (vo, c.v, c.v_scale)):
        with np.errstate(over="ignore"):
            want = mx_values(t, sc)[0, 0].astype(np.float32)
        g = got.cpu().numpy()[:, 0]
        assert np.array_equal(np.isnan(want), np.isnan(g))
        assert np.array_equal(want[~np.isnan(want)], g[~np.isnan(want)])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D,R,inter", [(48, 8, 128, 128, False), (4, 2, 64, 32, True), (5, 5, 256, 256, False),
                                              (16, 1, 128, 0, False)])
def test_norm_rotation_into_four_bits(act, hq, hkv, D, R, inter):
    say(f"norm, rotation into 4 bits {act} {hq}/{hkv} D={D} R={R}")
    T, P = 60, 16
    cfg = beam.AttnCfg(hq, hkv, D, R, inter, 0, P)
    q, k, v, pos, gq, gk, f = base.rope_inputs(cfg, T, act, 5, 8)
    c = beam.kv_cache(cfg, 5, beam.BEAM_MXFP4, DEV)
    qo = torch.empty((T, hq, D), dtype=base.ACT[act], device=DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, qo, c, f, gq, gk)
    ko, vo = (torch.empty((T, hkv, D), device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, i32([[0, 1, 2, 3]]), i32([0, T]), ko, vo)
    base.check_rows("q", qo, base.rope_ref(cfg, q, gq, pos, f, True), HALF[base.ACT[act]])
    s, e = oracle.quantize_mx_fp4(f64(v))
    assert np.array_equal(f64(vo), e * np.repeat(np.exp2(s.astype(float) - 127), 32, -1))
    want = base.rope_ref(cfg, k, gk, pos, f, False).reshape(T, hkv, -1, 32)
    got = f64(ko).reshape(want.shape)
    err = 2.0 ** -18 * np.abs(want).max((-1, -2), keepdims=True)
    top = np.abs(want).max(-1, keepdims=True)
    ok = np.zeros(want.shape[:-1], bool)
    for t in (top - err, top + err):                            # either scale, near a power of two
        step = np.exp2(np.floor(np.log2(t)) - 2)
        y = np.abs(want) / step
        half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
        half = np.where(y > 6, np.maximum(half, y - 6), half)
        half = np.maximum(half, np.where(np.abs(y - 2) < 0.25, 0.5, np.where(np.abs(y - 4) < 0.5, 1.0, 0)))
        ok |= (np.abs(got - want) <= half * step + err).all(-1)
    assert ok.all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_a_prompt_in_chunks_then_decoded(kind, window, sinks):
    """Prompts through norm, rotation, cache and attention in chunks, then tokens one at a time beside another
    prompt's chunk: what the sublayer computes from the cached rows at each step."""
    say(f"sublayer {kind} window={window}")
    P, hq, hkv, D = 16, 12, 2, 64
    cfg = beam.AttnCfg(hq, hkv, D, D, False, window, P, softmax_scale=0.125, sinks=sinks)
    act = act_of(kind)
    c = poisoned(cfg, 30, kind)
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(DEV)
    gq, gk = (torch.full((D,), x, dtype=act, device=DEV) for x in (1.5, 1.0))
    width = 8
    table = np.random.default_rng(3).permutation(30)[:3 * width].reshape(3, width).astype(np.int32)
    lens = [0, 0, 0]
    for step, new in enumerate([[50, 3, 0], [21, 1, 30], [1, 1, 40], [1, 1, 1], [1, 1, 1]]):
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(off[-1])
        pos, slots = [], []
        for b, n in enumerate(new):
            for i in range(n):
                p = lens[b] + i
                pos.append(p)
                slots.append(int(table[b, p // P]) * P + p % P)
            lens[b] += n
        qkv = torch.randn((T, (hq + 2 * hkv) * D), generator=gen(100 + step), device=DEV).to(act)
        if max(new) > 1:
            bufs = beam.attn_prompt_buffers(cfg, 3, T, 128, act, keep_lse=True)
            beam.attn_prompt_layer(cfg, qkv, i32(pos), i32(slots), c, i32(table), i32(off), i32(lens), 128, bufs, f, gq,
                                   gk)
        else:
            bufs = beam.attn_buffers(cfg, 3, 128, act, keep_lse=True)
            beam.attn_layer(cfg, qkv, i32(pos), i32(slots), c, i32(table), i32(lens), 128, bufs, f, gq, gk)
        torch.cuda.synchronize()
        # the cached rows as they are
        ko, vo = (torch.empty((30 * P, hkv, D), device=DEV) for _ in range(2))
        beam.beam_moe_kv_read(cfg, c, torch.arange(30, dtype=torch.int32, device=DEV)[None], i32([0, 30 * P]), ko, vo)
        vals = [np.nan_to_num(f64(x)).reshape(30, P, hkv, D).transpose(0, 2, 1, 3) for x in (ko, vo)]
        ro, rl, eo, el = prompt_ref(cfg, kind, bufs.q, *vals, table, off, lens, 30)
        assert (np.abs(f64(bufs.out) - ro) <= eo).all(), step
        assert (np.abs(f64(bufs.lse) - rl) <= el).all(), step


# ------------------------------------------------------------------ refusals

def test_bad_prompt_calls_are_refused():
    cfg = beam.AttnCfg(8, 2, 128, 0, False, 0, 16)
    c, _ = filled(cfg, 10, "bf16", 1)
    c4, _ = filled(cfg, 10, "fp4", 1)
    f4 = beam.AttnCfg(8, 2, 256, 0, False, 0, 16)
    q, out = (torch.zeros((5, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, off, lens = i32([[0, 1, 2], [3, 4, 5]]), i32([0, 2, 5]), i32([30, 40])
    ws = beam.attn_prompt_workspace(cfg, 2, 5, 48)
    good = dict(cfg=cfg, q=q, cache=c, page_table=table, q_offsets=off, seq_lens=lens, max_len=48, out=out, ws=ws)
    beam.beam_moe_attn_prompt(**good)
    for bad in (dict(q=q.float()), dict(q=q[:, :7]), dict(q=q.cpu()), dict(q=q.transpose(1, 2)), dict(out=out[:4]),
                dict(out=out.float()), dict(page_table=table[:1]), dict(page_table=table.long()),
                dict(q_offsets=off[:2]), dict(q_offsets=off.long()), dict(q_offsets=off.cpu()), dict(seq_lens=lens[:1]),
                dict(max_len=-1), dict(max_len=(1 << 30) + 1), dict(max_len=1 << 32), dict(out=q),
                dict(lse=torch.empty((5, 7), device=DEV)), dict(lse=torch.empty((5, 8), device=DEV).double()),
                dict(cfg=beam.AttnCfg(8, 2, 128, 0, False, 0, 32)), dict(cfg=f4, cache=c4),
                dict(cfg=beam.AttnCfg(8, 2, 128, 0, False, 0, 16, sinks=-1)),
                dict(cfg=beam.AttnCfg(8, 2, 128, 0, False, 0, 16, sinks=(1 << 30) + 1)),
                dict(cache=filled(cfg, 4, "f32", 1)[0])):
        with pytest.raises((ValueError, beam.BeamError)):
            beam.beam_moe_attn_prompt(**dict(good, **bad))
    # a workspace that is too small, where one is needed
    assert beam.lib().beam_moe_attn_prompt_workspace_bytes(cfg.c(), 0, 2, 5, 5000) > 256
    with pytest.raises(beam.BeamError):
        beam.beam_moe_attn_prompt(**dict(good, max_len=5000, ws=ws[:256]))
    with pytest.raises(beam.BeamError):
        beam.beam_moe_attn_prompt(**dict(good, max_len=5000, ws=None))
    # and nothing to do
    beam.beam_moe_attn_prompt(**dict(good, q=q[:0], out=out[:0], q_offsets=i32([0, 0, 0])))
    beam.beam_moe_attn_prompt(**dict(good, page_table=table[:0], q_offsets=off[:1], seq_lens=lens[:0]))


def test_bad_four_bit_caches_are_refused():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    good = (u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 4))
    cfg = beam.AttnCfg(4, 2, 128, 0, False, 0, 16)
    beam.KVCache(*good).c(cfg, 0)
    for i, t in ((1, u8(3, 2, 16, 32)), (2, u8(3, 2, 16, 2)), (3, u8(3, 2, 16)), (3, torch.zeros((3, 2, 16, 4), device=DEV)),
                 (3, None), (0, u8(3, 2, 16, 128)[..., ::2])):
        with pytest.raises(ValueError):
            beam.KVCache(*(t if j == i else x for j, x in enumerate(good)))
    with pytest.raises(ValueError):
        beam.KVCache(*good).c(beam.AttnCfg(4, 2, 64, 0, False, 0, 16), 0)


@pytest.mark.parametrize("fn", ["prompt", "decode"])
def test_native_marshalling_is_the_python_one(fn, monkeypatch):
    cfg = beam.AttnCfg(8, 2, 128, 0, False, 20, 16, sinks=3)
    for kind in ("bf16", "fp4"):
        c, _ = filled(cfg, 10, kind, 1)
        table, off, lens = i32([[0, 1, 2], [3, 4, 5]]), i32([0, 1, 2]), i32([30, 40])
        q = torch.randn((2, 8, 128), generator=gen(4), device=DEV).to(torch.bfloat16)
        outs = []
        for native in (True, False):
            with monkeypatch.context() as m:
                if native:
                    name = "attn_prompt" if fn == "prompt" else "attn_decode_sinks"
                    assert beam._native or beam._marshal()
                    assert hasattr(beam._native, name)
                    m.setattr(beam, "_launch", None)            # the Python way would fail
                else:
                    m.setattr(beam, "_native", False)
                out, lse = torch.empty_like(q), torch.empty((2, 8), device=DEV)
                if fn == "prompt":
                    beam.beam_moe_attn_prompt(cfg, q, c, table, off, lens, 48, out,
                                              beam.attn_prompt_workspace(cfg, 2, 2, 48), lse)
                else:
                    beam.beam_moe_attn_decode(cfg, q, c, table, lens, 48, out, beam.attn_workspace(cfg, 2, 48), lse)
                outs.append((out, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
