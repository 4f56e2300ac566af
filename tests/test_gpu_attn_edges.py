"""GPU tests of the attention sublayer where a wrong answer is easy to miss:
weights of the second product, values that are infinite.

Tolerances follow test_gpu_attn.py's head (h, u, A, e and n as there).  With a
bf16 or e4m3 cache a probability enters the second product as two bf16 parts:
its leading 8 bits, which leave less than 2^-7 of it, and the rounded rest, so
it is off by 2^-8 * 2^-7 = 2^-15 at most (and by 2^-24 where the rest is
nothing), in place of that head's h(bf16).
"""

import numpy as np
import pytest
import torch

import oracle
import test_gpu_attn as base
from parity_util import say

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ weights of the second product

@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (16, 1, 64), (40, 1, 128), (6, 2, 256)])
def test_equal_values_come_back(kind, hq, hkv, D):
    """The mean of equal values is that value, whatever the weights are: here
    scores that are equal, but not equal to the ones before them (which set
    the reference of the softmax)."""
    say(f"equal values {kind} {hq}/{hkv} D={D}")
    n, first = 2048, 128                                   # 128 tokens: one step of a workgroup
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, 0, 64, softmax_scale=1.0)
    c = beam.kv_cache(cfg, n // 64, base.KIND[kind])
    scale = 0.5 if kind == "fp8" else 1.0
    c.k.copy_(torch.zeros(c.k.shape, device=DEV))
    c.k[first // 64:, :, :, 0] = torch.full((), 1 / scale, device=DEV).to(c.k.dtype)
    c.v.copy_(torch.full(c.v.shape, 1 / scale, device=DEV))
    if kind == "fp8":
        c.k_scale.fill_(scale)
        c.v_scale.fill_(scale)
    q = torch.zeros((1, hq, D), device=DEV)
    q[0, :, 0] = torch.linspace(0.0037, 0.75, hq, device=DEV)
    q = q.to(base.ACT["f32" if kind == "f32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty((1, hq), device=DEV)
    table = torch.arange(n // 64, dtype=torch.int32, device=DEV)[None]
    # far fewer tokens expected: they all go to one workgroup
    beam.beam_moe_attn_decode(cfg, q, c, table, i32([n]), 100, out, None, lse)
    torch.cuda.synchronize()
    got = out.double()
    say(f"  off by {(got - 1).abs().max().item():.2e}")
    if kind == "f32":
        assert ((got - 1).abs() <= (n / 32 + 64) * 2.0 ** -24).all()
    else:                                                   # 2^-15 is far below half a step, 2^-9
        assert (got == 1).all()
    ref = torch.log(first + (n - first) * q[0, :, 0].double().exp())
    assert ((lse[0].double() - ref).abs() <= (n / 32 + 64 + ref) * 2.0 ** -24).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,D", [(48, 8, 128), (4, 4, 64), (64, 1, 128), (16, 1, 256)])
@pytest.mark.parametrize("window", [0, 100])
def test_decode_to_the_last_rounding(kind, hq, hkv, D, window):
    """The result is one rounding to bf16 away from the formula's."""
    say(f"last rounding {kind} {hq}/{hkv} D={D} window={window}")
    lens, P = [1, 33, 300, 900], 32
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5)
    n_pages = sum(-(-n // P) for n in lens) + 1
    c, (k, v) = base.filled(cfg, n_pages, kind, 17)
    table = base.tables(lens, P, n_pages, 5)
    q = (2 * torch.randn((len(lens), hq, D), generator=base.gen(3), device=DEV)).bfloat16()
    out = torch.empty_like(q)
    beam.beam_moe_attn_decode(cfg, q, c, torch.tensor(table, device=DEV), i32(lens), 900, out,
                              beam.attn_workspace(cfg, len(lens), 900))
    torch.cuda.synchronize()
    u, over = base.U, -1.0
    for b, n in enumerate(lens):
        toks = range(max(0, n - window) if window else 0, n)
        kr, _ = oracle.cached_rows(k, table[b], toks, n_pages)
        vr, _ = oracle.cached_rows(v, table[b], toks, n_pages)
        qb = base.f64(q[b]).reshape(hkv, hq // hkv, D)
        ref, _, mag = oracle.decode_attention(qb, kr, vr, cfg.softmax_scale)
        Z = cfg.softmax_scale * max((np.abs(qb[h]) @ np.abs(kr[:, h]).T).max() for h in range(hkv))
        bound = (2.0 ** -15 + 2 * u + 2 * (D / 4 + 8) * u * Z + (len(kr) / 32 + 64) * u) * mag + 2.0 ** -8 * np.abs(ref)
        over = max(over, (np.abs(base.f64(out[b]).reshape(ref.shape) - ref) - bound).max())
    say(f"  over the bound by {over:.2e}")
    assert over <= 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_infinite_values(kind):
    """An infinite value that is seen makes its own column infinite."""
    cfg = beam.AttnCfg(4, 2, 64, 0, False, 0, 16, softmax_scale=0.5)
    c, _ = base.filled(cfg, 4, kind, 2)
    q = torch.randn((1, 4, 64), generator=base.gen(4), device=DEV).to(base.ACT[kind])
    q[0, 0] = 0                                             # equal scores: weights of 1
    c.v[1, 0, 3, 5], c.v[2, 0, 9, 6] = float("inf"), float("-inf")
    out = torch.empty_like(q)
    beam.beam_moe_attn_decode(cfg, q, c, i32([[0, 1, 2, 3]]), i32([60]), 60, out, None)
    torch.cuda.synchronize()
    assert torch.isposinf(out[0, :2, 5]).all() and torch.isneginf(out[0, :2, 6]).all()
    assert torch.isfinite(out).sum() == out.numel() - 4


# ------------------------------------------------------------------ failures

def test_a_failed_launch_is_not_made_again(monkeypatch):
    """A call that the library answers with a HIP failure raises, and neither
    it nor the checks behind the marshalling call the library again: here the
    norm in place, which a second call would apply twice."""
    import ctypes
    from expert_routed_ffn_amd import _bind
    cfg = beam.AttnCfg(4, 2, 64, 32, False, 0, 16)
    q, k, _, pos, gq, gk, f = base.rope_inputs(cfg, 3, "bf16", 8)
    q, k = q.contiguous(), k.contiguous()
    kept = q.clone(), k.clone()
    calls = []
    fn = beam.lib().beam_moe_qk_norm_rope
    failing = ctypes.CFUNCTYPE(ctypes.c_int32, *fn.argtypes)(lambda *a: calls.append(a) or 4)
    at = [ctypes.cast(failing, ctypes.c_void_p).value] + [
        ctypes.cast(getattr(beam.lib(), "beam_moe_" + n), ctypes.c_void_p).value
        for n in ("qk_norm_rope_cache", "kv_write", "kv_read", "attn_decode")]
    _bind.bind(torch.Tensor.__dlpack_c_exchange_api__, int(q.__dlpack_device__()[0]), *at)
    monkeypatch.setattr(beam, "_native", _bind)
    try:
        with pytest.raises(RuntimeError):
            beam.beam_moe_qk_norm_rope(cfg, q, k, pos, q, k, f, gq, gk)
    finally:
        monkeypatch.undo()
        beam._native = None                                 # bound to the library anew
    torch.cuda.synchronize()
    assert len(calls) == 1 and torch.equal(q, kept[0]) and torch.equal(k, kept[1])
    beam.beam_moe_qk_norm_rope(cfg, q, k, pos, q, k, f, gq, gk)
    torch.cuda.synchronize()
    assert not torch.equal(q, kept[0])


def hip_runtime():
    """The HIP runtime that this process has loaded."""
    import ctypes
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64" in line}
    assert len(paths) == 1, paths
    return ctypes.CDLL(paths.pop())


@pytest.mark.parametrize("name", base.CALLS)
@pytest.mark.parametrize("native", [True, False])
def test_an_earlier_error_is_not_this_calls(name, native):
    """An error that an unrelated HIP call left (a device that is not there)
    neither fails a call that runs nor makes it run twice."""
    hip = hip_runtime()
    s = base.binding_state()
    s["k"], s["q"] = s["k"].contiguous(), s["q"].contiguous()
    if name == "rope":
        s["ko"], s["qo"] = s["k"], s["q"]                   # in place
    kw = {} if native else {"stream": torch.cuda.current_stream()}
    sides = (s["cache"].k, s["cache"].v, s["cache"].k_scale, s["cache"].v_scale)
    touched = [s[r] for r in base.RESULTS[name]] + list(sides)
    start = [t.clone() for t in touched]
    base.CALLS[name](s, **kw)
    torch.cuda.synchronize()
    want = [t.clone() for t in touched]
    for t, u in zip(touched, start):
        t.copy_(u)
    torch.cuda.synchronize()
    assert hip.hipSetDevice(1 << 10) != 0
    try:
        base.CALLS[name](s, **kw)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    for t, u in zip(touched, want):
        assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))


# ------------------------------------------------------------------ read back

@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("hkv,D,N", [(64, 128, 90), (256, 64, 70), (33, 256, 41), (1, 64, 3000), (256, 256, 5)])
def test_read_back_of_many_and_few_heads(kind, hkv, D, N):
    """Rows that take a workgroup several turns, and as many rows as it takes."""
    cfg = beam.AttnCfg(hkv, hkv, D, 0, False, 0, 16)
    n_pages = -(-N // 16) + 2
    c, (k, v) = base.filled(cfg, n_pages, kind, 5)
    table = base.tables([N], 16, n_pages, 2)
    ko, vo = (torch.full((N + 2, hkv, D), 3.0, device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, torch.tensor(table, device=DEV), i32([0, N]), ko, vo)
    torch.cuda.synchronize()
    t = np.arange(N)
    for got, ref in ((ko, k), (vo, v)):
        assert np.array_equal(base.f64(got[:N]), ref[table[0, t // 16], :, t % 16].astype(np.float32))
        assert (got[N:] == 3).all()


# ------------------------------------------------------------------ e4m3 rows

def awkward_rows(T, hkv, D, act, seed):
    """Rows with zeros of both signs in them, of both signs only, of extreme
    sizes (whose division goes another way), of values at the codes' borders."""
    g = base.gen(seed)
    x = torch.randn((T, hkv, D), generator=g, device=DEV)
    x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.2, torch.zeros_like(x), x)
    x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.5, -x, x)
    x[3::11] *= 1e-30
    x[5::11] *= 1e30
    x[7::11, 0] *= 0
    x[8::11] = torch.arange(D, device=DEV) * (448.0 / 256)
    x[9::11, :, ::2] *= 2.0 ** -12
    return x.to(base.ACT[act])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("special", [False, True])
def test_cache_codes_are_the_quantisers(D, special):
    """Codes and scales of a stored row are, byte for byte, those of
    beam_moe_quantize_fp8, whatever rows stand beside it: signs of zeros,
    rows of extreme sizes, NaN and infinities too."""
    T, hkv = 66, 3
    x = awkward_rows(T, hkv, D, "bf16", D)
    if special:
        x[0, 0, 3], x[1, 1, 5], x[2, 2, 7], x[4, 0, 9] = (float(s) for s in ("nan", "inf", "-inf", "nan"))
        x.view(torch.int16)[4, 0, 9] = -64                  # a NaN with its sign set
    cfg = beam.AttnCfg(hkv, hkv, D, 0, False, 0, 16)
    c = beam.kv_cache(cfg, 5, beam.BEAM_FP8_E4M3)
    beam.beam_moe_kv_write(cfg, x, x.flip(0), torch.arange(T, dtype=torch.int32, device=DEV), c)
    wide = torch.zeros((T * hkv, 256), dtype=torch.bfloat16, device=DEV)     # zeros behind a row change nothing of it
    wide[:, :D] = x.view(T * hkv, D)
    codes = torch.empty((T * hkv, 256), dtype=torch.uint8, device=DEV)
    scale = torch.empty(T * hkv, device=DEV)
    beam.beam_moe_quantize_fp8(beam.LayerCfg(hidden=256), wide, codes, scale)
    torch.cuda.synchronize()
    want, ws = codes[:, :D].view(T, hkv, D), scale.view(T, hkv)
    t = torch.arange(T, device=DEV)
    for side, sc, order in ((c.k, c.k_scale, t), (c.v, c.v_scale, t.flip(0))):
        got = side.view(torch.uint8)[t // 16, :, t % 16]
        assert torch.equal(sc[t // 16, :, t % 16].view(torch.int32), ws[order].view(torch.int32))
        bad = torch.nonzero(got != want[order])
        say(f"  D={D}: {len(bad)} codes differ")
        assert len(bad) == 0
    assert special or (want[:, :, :] == 0x80).any()         # there are zeros below zero


@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_codes_of_fp32_rows(D):
    """fp32 rows: each code is e4m3 of the correctly rounded fp32 quotient."""
    T, hkv = 660, 3
    x = awkward_rows(T, hkv, D, "f32", D + 1)
    # a scale of 2 - 2^-23, whose reciprocal lies next to the middle of two
    # floats: 2^-9 / scale is just above 2^-10, the middle of codes 0 and 1
    x[0, 0] = 0
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = 896 - 2.0 ** -14, 2.0 ** -9, -2.0 ** -9
    cfg = beam.AttnCfg(hkv, hkv, D, 0, False, 0, 64)
    c = beam.kv_cache(cfg, 11, beam.BEAM_FP8_E4M3)
    beam.beam_moe_kv_write(cfg, x, x, torch.arange(T, dtype=torch.int32, device=DEV), c)
    torch.cuda.synchronize()
    h = x.cpu().numpy()
    top = np.abs(h).max(-1)
    s = np.where(top > 0, top / np.float32(448), np.float32(1))
    want = torch.tensor(h / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert s[0, 0] == 2 - 2.0 ** -23 and want[0, 0, 1] == 1 and want[0, 0, 2] == 0x81
    t = torch.arange(T, device=DEV)
    for side, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert np.array_equal(sc[t // 64, :, t % 64].cpu().numpy(), s)
        assert torch.equal(side.view(torch.uint8)[t // 64, :, t % 64].cpu(), want)


def test_rows_of_the_least_floats():
    """A row so small that its scale would round to zero is stored as zeros."""
    cfg = beam.AttnCfg(2, 2, 64, 0, False, 0, 16)
    x = torch.zeros((4, 2, 64), device=DEV)
    least = 2.0 ** -149
    x[0, 0, 3], x[0, 1, 5], x[1, 0, 1], x[1, 1, 9] = least, -least, 224 * least, 225 * least
    x[2] = -0.0
    c = base.poisoned(cfg, 1, "fp8")
    beam.beam_moe_kv_write(cfg, x, x, torch.arange(4, dtype=torch.int32, device=DEV), c)
    ko, vo = (torch.empty((4, 2, 64), device=DEV) for _ in range(2))
    beam.beam_moe_kv_read(cfg, c, i32([[0]]), i32([0, 4]), ko, vo)
    torch.cuda.synchronize()
    want_s = [[1, 1], [1, least], [1, 1], [1, 1]]           # 224/448 is a tie, and goes to 0
    for got, sc in ((ko, c.k_scale), (vo, c.v_scale)):
        assert sc[0, :, :4].t().double().tolist() == want_s
        assert torch.isfinite(got).all()
        assert ((got.double() - x.double()).abs() <= 224 * least).all()
        assert got[1, 1, 9].item() == 224 * least           # code 224, the nearest to 225


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("max_len", [(1 << 32) + 32, 1 << 32, -(1 << 32), (1 << 31), (1 << 30) + 1, -1])
@pytest.mark.parametrize("native", [True, False])
def test_lengths_to_expect_beyond_the_limit(max_len, native):
    """Refused, not taken modulo 2^32."""
    s = base.binding_state()
    s["out"].fill_(3.0)
    kw = {} if native else {"stream": torch.cuda.current_stream()}
    with pytest.raises((ValueError, beam.BeamError)):
        beam.beam_moe_attn_decode(s["cfg"], s["qo"], s["cache"], s["table"], s["lens"], max_len, s["out"], s["ws"],
                                  s["lse"], **kw)
    torch.cuda.synchronize()
    assert (s["out"] == 3).all()


# ------------------------------------------------------------------ long sequences among many

def exact_decode(cfg, q, vals, table, lens):
    """fp64 (out, magnitude, lse) on the GPU, and the bound on a score."""
    B, hq, D = q.shape
    hkv, P = cfg.n_kv_heads, cfg.page_size
    out, mag = (torch.zeros((B, hq, D), dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((B, hq), -float("inf"), dtype=torch.float64, device=DEV)
    Z = torch.zeros(B, dtype=torch.float64, device=DEV)
    k, v = vals
    for b, n in enumerate(lens):
        if n == 0:
            continue
        t = torch.arange(max(0, n - cfg.window) if cfg.window else 0, n, device=DEV)
        page = table[b].long()[t // P]
        kr, vr = (x[page, :, t % P].transpose(0, 1).contiguous() for x in (k, v))          # [hkv, n, D]
        qb = q[b].double().view(hkv, hq // hkv, D)
        z = cfg.softmax_scale * torch.matmul(qb, kr.transpose(1, 2).contiguous())
        w = torch.softmax(z, -1)
        out[b], mag[b] = (torch.matmul(w, x).view(hq, D) for x in (vr, vr.abs()))
        lse[b] = torch.logsumexp(z, -1).view(hq)
        Z[b] = cfg.softmax_scale * torch.matmul(qb.abs(), kr.abs().transpose(1, 2).contiguous()).max()
    return out, mag, lse, Z


def pages_for(lens, P, n_pages, seed):
    """Any pages, shared by all."""
    width = max(1, -(-max(lens) // P))
    return torch.randint(0, n_pages, (len(lens), width), generator=base.gen(seed), device=DEV, dtype=torch.int32)


MANY = {
    "long first": lambda r: [20001] + [int(x) for x in r.integers(0, 300, 90)],
    "long last": lambda r: [int(x) for x in r.integers(0, 300, 300)] + [33000],
    "long in the middle, empty ones": lambda r: [0] * 40 + [5000, 0, 4097, 0, 4096] + [0] * 40,
    "all long": lambda r: [int(x) for x in r.integers(4000, 9000, 70)],
    "two": lambda r: [9000, 130],
    "most": lambda r: [int(x) for x in r.integers(0, 40, 4094)] + [8200],
    "one more": lambda r: [int(x) for x in r.integers(0, 40, 4095)] + [8200],
    "all empty": lambda r: [0] * 100,
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("name,hq,hkv,D,window,max_len", [
    ("long first", 8, 8, 128, 0, 131072), ("long first", 48, 8, 64, 10000, 1 << 20), ("long last", 16, 8, 128, 0, 131072),
    ("long last", 40, 2, 256, 0, 1 << 20), ("long in the middle, empty ones", 16, 16, 64, 0, 131072),
    ("all long", 64, 64, 64, 0, 131072), ("all long", 64, 1, 128, 0, 1 << 20), ("two", 64, 1, 64, 0, 1 << 30),
    ("most", 2, 2, 64, 0, 131072), ("one more", 2, 2, 64, 0, 131072), ("all empty", 8, 8, 64, 0, 131072),
])
def test_decode_of_listed_parts(kind, name, hq, hkv, D, window, max_len):
    """Batches whose parts are listed: one or all long, at any place, more
    parts than are listed at their usual size, query heads in several groups."""
    say(f"listed parts {kind} {name} {hq}/{hkv} D={D} expected {max_len}")
    lens = MANY[name](np.random.default_rng(7))
    B, P, n_pages = len(lens), 256, 9
    cfg = beam.AttnCfg(hq, hkv, D, 0, False, window, P, softmax_scale=D ** -0.5)
    c, vals = base.filled(cfg, n_pages, kind, 31)
    vals = [torch.tensor(x, device=DEV) for x in vals]
    table = pages_for(lens, P, n_pages, 3)
    q = (2 * torch.randn((B, hq, D), generator=base.gen(5), device=DEV)).to(base.ACT["f32" if kind == "f32" else "bf16"])
    out, lse = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV), torch.full((B, hq), 9.0, device=DEV)
    ws = beam.attn_workspace(cfg, B, max_len)
    ws.fill_(0xFF)                                         # its contents do not matter
    beam.beam_moe_attn_decode(cfg, q, c, table, i32(lens), max_len, out, ws, lse)
    torch.cuda.synchronize()
    ro, mag, rl, Z = exact_decode(cfg, q, vals, table, lens)
    u, n = base.U, torch.tensor(lens, device=DEV).double()
    e, cu = (D / 4 + 8) * u * Z, (n / 32 + 64) * u
    weight = 0.0 if kind == "f32" else 2.0 ** -15 + 2 * u
    bound = (weight + 2 * e + cu)[:, None, None] * mag + base.HALF[q.dtype] * ro.abs()
    over = ((out.double() - ro).abs() - bound).max().item()
    say(f"  over the bound by {over:.2e}")
    assert over <= 0
    some = n > 0
    assert torch.isneginf(lse[~some]).all() and (out[~some] == 0).all()
    assert ((lse.double() - rl).abs()[some] <= ((e + cu)[:, None] + u * rl.abs())[some]).all()
    again = torch.empty_like(out)
    beam.beam_moe_attn_decode(cfg, q, c, table, i32(lens), max_len, again, ws, lse)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def test_listed_parts_in_a_graph_and_on_two_streams():
    """A captured call replayed with other lengths, and two calls at once with
    a workspace each, give the eager bits."""
    cfg = beam.AttnCfg(16, 8, 128, 0, False, 0, 64)
    B, n_pages, max_len = 80, 30, 131072
    c, _ = base.filled(cfg, n_pages, "fp8", 3)
    r = np.random.default_rng(5)
    batches = [[int(x) for x in r.integers(0, 500, B)] for _ in range(3)]
    batches[0][79], batches[1][0], batches[2][40] = 12000, 9000, 1
    table = pages_for([12000] * B, 64, n_pages, 1)
    q = torch.randn((B, 16, 128), generator=base.gen(2), device=DEV).bfloat16()
    ws = [beam.attn_workspace(cfg, B, max_len) for _ in range(2)]
    out, lens = torch.empty_like(q), i32(batches[0])
    eager = []
    for x in batches:
        lens.copy_(i32(x))
        beam.beam_moe_attn_decode(cfg, q, c, table, lens, max_len, out, ws[0])
        eager.append(out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beam.beam_moe_attn_decode(cfg, q, c, table, lens, max_len, out, ws[0])
    for i in (0, 1, 2, 1, 0):
        lens.copy_(i32(batches[i]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, ls = [torch.empty_like(q) for _ in range(2)], [i32(batches[i]) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            beam.beam_moe_attn_decode(cfg, q, c, table, ls[i], max_len, outs[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], eager[i])


# ------------------------------------------------------------------ norm

def test_norm_factor_is_one_rounding_off():
    """1 / sqrt(mean(x^2) + eps), seen through rows of a power of two so small
    that eps alone counts: half a unit in the last place (and 2^-10 of one)."""
    g = np.random.default_rng(8)
    x = torch.full((1, 1, 64), 2.0 ** -30, device=DEV)
    one, pos = torch.ones(64, device=DEV), i32([0])
    eps = np.exp2(g.uniform(-8, 8, 400)).astype(np.float32)
    outs = []
    for e in eps:
        cfg = beam.AttnCfg(1, 1, 64, 0, False, 0, 16, rms_eps=float(e))
        q, k = torch.empty_like(x), torch.empty_like(x)
        beam.beam_moe_qk_norm_rope(cfg, x, x, pos, q, k, None, one, one)
        outs.append(torch.stack([q[0, 0], k[0, 0]]))
    got = base.f64(torch.stack(outs)) * 2.0 ** 30
    assert (got == got[:, :1, :1]).all()
    want = 1 / np.sqrt(eps.astype(np.float64))
    unit = 2.0 ** (np.floor(np.log2(want)) - 23)
    off = np.abs(got[:, 0, 0] - want) / unit
    say(f"  up to {off.max():.4f} units off")
    assert (off <= 0.5 + 2.0 ** -10).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_norm_of_extreme_rows(act):
    """No epsilon: rows of zeros give NaN (0/0), rows far from 1 the formula's
    values as long as their squares' mean is a normal float, and stay finite
    beyond."""
    cfg = beam.AttnCfg(6, 1, 64, 0, False, 0, 16, rms_eps=0.0)
    q = torch.randn((1, 6, 64), generator=base.gen(6), device=DEV)
    for h, size in enumerate((0.0, 1e-17, 1e-10, 1.0, 1e10, 1e17)):
        q[0, h] *= size
    q = q.to(base.ACT[act])
    k = q[:, 3:4].contiguous() * 2.0 ** 66                  # squares overflow: a factor of 0
    one = torch.ones(64, dtype=q.dtype, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beam.beam_moe_qk_norm_rope(cfg, q, k, i32([0]), qo, ko, None, one, one)
    torch.cuda.synchronize()
    assert torch.isnan(qo[0, 0]).all() and (ko == 0).all()
    base.check_rows("q", qo[:, 1:], base.rope_ref(cfg, q[:, 1:], one, i32([0]), None, False), base.HALF[q.dtype])


# ------------------------------------------------------------------ calls that the other tests leave out

@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [0, 700])
def test_listed_parts_with_bad_pages_and_lengths(kind, window):
    """Lengths below zero and beyond the table, pages outside the cache."""
    P, n_pages, B = 64, 20, 70
    cfg = beam.AttnCfg(16, 8, 64, 0, False, window, P)
    c, vals = base.filled(cfg, n_pages, kind, 5)
    r = np.random.default_rng(2)
    table = r.integers(0, n_pages, (B, 90)).astype(np.int32)
    lens = r.integers(0, 200, B)
    lens[[0, 3, 20, 69]] = [-5, 1 << 30, 5760, -(1 << 31)]
    lens[[7, 8]] = [(1 << 31) - 1, 5000]
    table[3, ::3], table[7, 10:], table[8], table[20, 64:] = -1, n_pages, 1 << 30, -(1 << 31)
    q = torch.randn((B, 16, 64), generator=base.gen(4), device=DEV).to(base.ACT["f32" if kind == "f32" else "bf16"])
    base.check_decode(cfg, q, c, vals, table, [int(x) for x in lens], 131072, f"bad pages, listed, window {window}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decode_of_as_many_key_value_heads_as_there_are(kind):
    lens = [1, 40, 300]
    cfg = beam.AttnCfg(256, 256, 64, 0, False, 0, 32, softmax_scale=0.125)
    c, vals = base.filled(cfg, 13, kind, 5)
    q = torch.randn((3, 256, 64), generator=base.gen(4), device=DEV).bfloat16()
    base.check_decode(cfg, q, c, vals, base.tables(lens, 32, 13, 2), lens, 300, "256 key-value heads")


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
def test_cached_form_in_place(kind):
    """The queries normed and rotated where they are, idle rows among them."""
    cfg = beam.AttnCfg(6, 2, 128, 64, False, 0, 16)
    q, k, v, pos, gq, gk, f = base.rope_inputs(cfg, 19, "bf16", 5)
    q = q.contiguous()
    slots = torch.arange(19, dtype=torch.int32, device=DEV)
    slots[4], slots[18] = -1, 1 << 20
    a, b = (base.poisoned(cfg, 2, kind) for _ in range(2))
    qo = torch.empty_like(q)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, qo, a, f, gq, gk)
    beam.beam_moe_qk_norm_rope_cache(cfg, q, k, v, pos, slots, q, b, f, gq, gk)
    torch.cuda.synchronize()
    assert torch.equal(q, qo)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_empty_calls():
    """No tokens, no sequences, no rows: nothing to do, and nothing refused."""
    cfg = beam.AttnCfg(4, 2, 64, 0, False, 0, 16)
    c, _ = base.filled(cfg, 2, "bf16", 1)
    kept = c.k.clone()
    q, k = (torch.empty((0, h, 64), dtype=torch.bfloat16, device=DEV) for h in (4, 2))
    none, table = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty((0, 3), dtype=torch.int32, device=DEV)
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        beam.beam_moe_qk_norm_rope(cfg, q, k, none, q.clone(), k.clone(), **kw)
        beam.beam_moe_qk_norm_rope_cache(cfg, q, k, k, none, none, q.clone(), c, **kw)
        beam.beam_moe_kv_write(cfg, k, k, none, c, **kw)
        beam.beam_moe_kv_read(cfg, c, table, i32([0]), k.clone(), k.clone(), **kw)
        beam.beam_moe_kv_read(cfg, c, i32([[0, 1]]), i32([0, 0]), k.clone(), k.clone(), **kw)
        ko, vo = (torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        beam.beam_moe_kv_read(cfg, c, table, i32([0]), ko, vo, **kw)
        beam.beam_moe_attn_decode(cfg, q, c, table, none, 100, q.clone(), None, **kw)
        torch.cuda.synchronize()
        assert torch.equal(c.k, kept) and (ko == 5).all() and (vo == 5).all()
