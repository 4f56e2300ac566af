"""Host-side checks of prompt attention, of sinks and of the 4-bit cache (no
GPU, no kernel is launched): invalid calls get the documented status before
anything is enqueued, empty calls are no-ops, and the native marshalling makes
a call once."""

import ctypes
import os

import pytest
import torch

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.skipif(not os.path.exists(beam.LIB_PATH), reason="library not built")

# never dereferenced: every call below fails validation first (or has nothing to do)
A = 1 << 32
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    return beam.lib()


def cfg(**kw):
    return beam.AttnCfg(**{"window": 0, **kw})


def kv(k=A * 10, v=A * 20, ks=None, vs=None, n=100, dt=beam.BEAM_BF16):
    return beam.BeamMoeKvCache(k, v, ks, vs, n, dt)


def fp4(**kw):
    return kv(**{**dict(ks=A * 30, vs=A * 31, dt=beam.BEAM_MXFP4), **kw})


def prompt(L, c=None, sinks=0, B=4, T=2000, q=A, qs=6144, dt=1, cache=None, tab=A * 2, mp=1024, off=A * 3, lens=A * 3,
           ml=60000, out=A * 4, lse=None, ws=None, wsb=0):
    return L.beam_moe_attn_prompt((c or cfg()).c(), sinks, B, T, q, qs, dt, cache if cache is not None else kv(), tab, mp,
                                  off, lens, ml, out, lse, ws, wsb, None)


def decode(L, c=None, sinks=0, B=4, q=A, qs=6144, dt=1, cache=None, tab=A * 2, mp=1024, lens=A * 3, ml=60000, out=A * 4,
           lse=None, ws=None, wsb=0):
    return L.beam_moe_attn_decode_sinks((c or cfg()).c(), sinks, B, q, qs, dt, cache if cache is not None else kv(), tab,
                                        mp, lens, ml, out, lse, ws, wsb, None)


@pytest.mark.parametrize("bad,want", [
    (dict(n_heads=0), 1), (dict(n_kv_heads=-3), 1), (dict(head_dim=96), 2), (dict(n_heads=50), 2),
    (dict(n_heads=65, n_kv_heads=1), 2), (dict(window=-1), 1), (dict(page_size=0), 1), (dict(page_size=48), 2),
    (dict(softmax_scale=0.0), 1), (dict(softmax_scale=float("nan")), 1),
])
def test_invalid_cfg(L, bad, want):
    c = cfg(**bad)
    assert prompt(L, c) == want and decode(L, c) == want
    assert L.beam_moe_attn_prompt_workspace_bytes(c.c(), 0, 4, 100, 4096) == 0
    assert L.beam_moe_attn_decode_sinks_workspace_bytes(c.c(), 0, 4, 4096) == 0
    assert L.beam_moe_attn_prompt(None, 0, 4, 8, A, 6144, 1, kv(), A, 8, A, A, 99, A * 4, None, None, 0, None) == 1


@pytest.mark.parametrize("bad,want", [
    (dict(sinks=-1), 1), (dict(sinks=(1 << 30) + 1), 1), (dict(B=-1), 1), (dict(B=(1 << 22) + 1), 1), (dict(mp=-1), 1),
    (dict(ml=-1), 1), (dict(ml=(1 << 30) + 1), 1), (dict(dt=2), 1), (dict(dt=9), 1), (dict(dt=0), 2), (dict(q=None), 1),
    (dict(q=A + 8), 1), (dict(qs=6140), 1), (dict(qs=6147), 1), (dict(out=None), 1), (dict(out=A), 1),
    (dict(out=A * 4 + 8), 1), (dict(tab=None), 1), (dict(tab=A + 2), 1), (dict(lens=None), 1), (dict(lens=A * 3 + 1), 1),
    (dict(lse=A + 1), 1), (dict(), 3), (dict(ws=A * 6, wsb=1024), 3), (dict(ws=A * 6 + 4, wsb=GB * 8), 3),
])
def test_arguments(L, bad, want):
    few = dict(T=8) if "ws" in bad or not bad else {}        # so few that a workspace is needed
    assert prompt(L, **bad, **few) == want
    assert decode(L, **bad) == want


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=(1 << 22) + 1), dict(off=None), dict(off=A + 2),
                                 dict(out=A + 6144 * 2 * 1999), dict(q=A * 4 + 16)])
def test_prompt_arguments(L, bad):
    assert prompt(L, **bad) == 1


def test_nothing_to_do(L):
    c = cfg()
    for B, T in ((0, 0), (0, 100), (5, 0)):
        assert L.beam_moe_attn_prompt(c.c(), 0, B, T, None, 0, 1, None, None, 0, None, None, 0, None, None, None, 0,
                                      None) == 0
    assert L.beam_moe_attn_decode_sinks(c.c(), 4, 0, None, 0, 1, None, None, 0, None, 0, None, None, None, 0, None) == 0


def test_dtypes(L):
    for f in (prompt, decode):
        assert f(L, cache=kv(dt=beam.BEAM_F32), dt=1) == 2                   # fp32 cache, bf16 queries
        assert f(L, cache=kv(dt=beam.BEAM_FP8_E4M3, ks=A, vs=A), dt=0) == 2
        assert f(L, cache=fp4(), dt=0) == 2
    assert prompt(L, cache=fp4(), dt=1, T=8) == 3 and decode(L, cache=fp4(), dt=1) == 3    # on to the workspace


@pytest.mark.parametrize("bad,want", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(k=A + 8), 1), (dict(v=A + 4), 1),
    (dict(ks=A + 2), 1), (dict(vs=A + 1), 1), (dict(n=0), 1), (dict(n=1 << 25), 2)])
def test_four_bit_caches(L, bad, want):
    c, cache = cfg(), fp4(**bad)
    assert prompt(L, cache=cache) == want and decode(L, cache=cache) == want
    assert L.beam_moe_kv_write(c.c(), 8, A, 1024, A * 2, 1024, 1, A * 3, cache, None) == want
    assert L.beam_moe_kv_read(c.c(), 4, 100, cache, A, 8, A * 2, None, A * 3, A * 4, 1, None) == want
    assert L.beam_moe_qk_norm_rope_cache(c.c(), 8, A, 8192, A + 12288, 8192, A + 14336, 8192, 1, A * 2, A * 2, A * 3,
                                         A * 3, A * 3, A * 4, cache, None) == want


def test_workspaces(L):
    def p(B, T, n, sinks=0, **kw):
        return L.beam_moe_attn_prompt_workspace_bytes(cfg(**kw).c(), sinks, B, T, n)

    def d(B, n, sinks=0, **kw):
        return L.beam_moe_attn_decode_sinks_workspace_bytes(cfg(**kw).c(), sinks, B, n)

    for w in (lambda B, n, sinks=0, **kw: p(B, B, n, sinks, **kw), d):
        assert w(-1, 10) == 0 and w(0, 10) == 0 and w(1, -1) == 0 and w(1, (1 << 30) + 1) == 0
        assert w(1, 100, -1) == 0 and w(1, 100, (1 << 30) + 1) == 0
        assert w(1, 1) == 0 and w(1, 131072) > 0
        assert w(1, 131072, 4, window=512) <= w(1, 131072)
        assert w(1, 131072, 100000, window=512) >= w(1, 131072, 4, window=512)
    assert d(4, 4096) == L.beam_moe_attn_workspace_bytes(cfg().c(), 4, 4096)
    assert p(1, 0, 100) == 0 and p(1, -1, 100) == 0 and p(1, (1 << 22) + 1, 100) == 0
    assert p(1, 16384, 16384) == 0                           # blocks enough
    assert p(65, 2112, 10240) > 0                            # some sequence may be one long block


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 32), (1, 300), (3, 17), (30, 30), (40, 320)])
def test_a_workspace_for_the_longest_serves_the_table(L, page, B, T):
    """max_len counts in whole pages, in the workspace and in the call."""
    for n in (1, 255, 256, 257, 1000, 1024, 1025, 5000, (1 << 30) - 1):
        c, whole = cfg(page_size=page), -(-n // page) * page
        need = L.beam_moe_attn_prompt_workspace_bytes(c.c(), 0, B, T, n)
        assert need == L.beam_moe_attn_prompt_workspace_bytes(c.c(), 0, B, T, whole)
        if need:
            assert prompt(L, c, B=B, T=T, ml=whole, ws=A * 6, wsb=need - 1) == 3


@pytest.mark.parametrize("hq,hkv", [(48, 8), (64, 1), (1, 1), (256, 256), (16384, 256)])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 1 << 22), (7, 5), (300, 300), (1 << 22, 1 << 22), (1 << 22, 1), (4096, 70000)])
@pytest.mark.parametrize("n,window,sinks", [(0, 0, 0), (1 << 30, 0, 0), (1 << 30, 1 << 20, 1 << 30), (1 << 30, 1, 1),
                                            (1 << 30, (1 << 31) - 1, 1 << 30)])
def test_every_call_is_launched_or_refused(L, hq, hkv, B, T, n, window, sinks):
    """Whatever the sizes, the workspace is a size that can be allocated, or
    the call is refused for its workgroups before the workspace is asked for."""
    c = cfg(n_heads=hq, n_kv_heads=hkv, head_dim=256, window=window)
    need = L.beam_moe_attn_prompt_workspace_bytes(c.c(), sinks, B, T, n)
    refused = (T * (hq // hkv) // 128 + B) * hkv >= 1 << 24
    assert need <= (1 << 24) * 128 * 260 * 4 or refused
    if need or refused:      # else it would be launched: not from here
        assert prompt(L, c, sinks, B, T, q=A, qs=hq * 256, out=A * 65536, ml=n) == (2 if refused else 3)


# ------------------------------------------------------------------ what the native marshalling makes of a call

ENTRIES = ("attn_decode_sinks", "attn_prompt")
OLD = ("qk_norm_rope", "qk_norm_rope_cache", "kv_write", "kv_read", "attn_decode")


def _bound(device, entries):
    from expert_routed_ffn_amd import _bind
    lib = beam.lib()
    at = [ctypes.cast(getattr(lib, "beam_moe_" + f), ctypes.c_void_p).value for f in OLD]
    _bind.bind(torch.Tensor.__dlpack_c_exchange_api__, device, *at, beam.BeamError)
    _bind.bind_more(*[ctypes.cast(e, ctypes.c_void_p).value for e in entries])
    return _bind


@pytest.fixture
def stub():
    lib, calls, keep = beam.lib(), [], []

    def make(status):
        for f in ENTRIES:
            types = getattr(lib, "beam_moe_" + f).argtypes
            keep.append(ctypes.CFUNCTYPE(ctypes.c_int32, *types)(lambda *a, f=f: calls.append((f, a)) or status))
        return _bound(1, keep), calls                       # tensors of the CPU
    yield make
    _bound(10, [getattr(lib, "beam_moe_" + f) for f in ENTRIES])     # no stub is called any more
    beam._native = None                                     # bound anew by the next call


def native_args(kind=beam.BEAM_BF16):
    c = beam.AttnCfg(2, 1, 64, 0, False, 0, 16, sinks=3)
    x, i = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    cache = beam.BeamMoeKvCache(pages.data_ptr(), pages.data_ptr(), None, None, 2, kind)
    table, off = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    args = (c._c, x, cache, pages, table, i, 32, x.clone(), None, None, 3)
    return {"attn_decode_sinks": args, "attn_prompt": (*args, off)}, (c, pages)


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_that_failed_in_hip_is_made_once(stub, name):
    (bind, calls), (args, keep) = stub(4), native_args()
    with pytest.raises(beam.BeamError) as e:
        getattr(bind, name)(*args[name])
    assert e.value.status == 4 and "beam_moe_" + name in str(e.value)
    assert [f for f, _ in calls] == [name]


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("status,want", [(0, True), (1, False), (2, False), (3, False)])
def test_refused_and_good_calls(stub, name, status, want):
    (bind, calls), (args, keep) = stub(status), native_args()
    assert getattr(bind, name)(*args[name]) is want
    assert [f for f, _ in calls] == [name]
    assert calls[0][1][1] == 3 and calls[0][1][2] == 3      # sinks, sequences


@pytest.mark.parametrize("name", ENTRIES)
def test_what_the_native_marshalling_leaves_to_python(stub, name):
    (bind, calls), (args, keep) = stub(0), native_args()
    fn, good = getattr(bind, name), args[name]
    assert fn(*good[:-1]) is False and fn(*[None] * len(good)) is False
    for at, other in ((1, "x"), (1, good[1].float()), (1, good[1][:, :, ::2]), (4, good[4].long()), (4, good[4].t()),
                      (4, good[4][0]), (5, good[5].long()), (5, good[5][:2]), (6, -1), (6, 1 << 40), (6, None), (7, None),
                      (7, good[7][:, :, :32]), (8, good[7]), (9, good[7]), (10, -1), (10, 1 << 40), (10, "x"), (10, None)):
        bad = list(good)
        bad[at] = other
        assert fn(*bad) is False, at
    if name == "attn_prompt":                               # offsets of another number of sequences
        for off in (good[11][:3], torch.zeros(6, dtype=torch.int32), None):
            assert fn(*good[:11], off) is False
    assert calls == []


def test_binding_refusals():
    for bad in (-(1 << 40), 1 << 32, 1 << 40):
        with pytest.raises(ValueError, match="sinks"):
            beam.AttnCfg(window=8, sinks=bad)
    c = beam.AttnCfg(n_heads=2, n_kv_heads=1, head_dim=64, rope_dim=0, window=8, sinks=2)
    with pytest.raises(ValueError):                         # not on a GPU
        beam.KVCache(torch.zeros((2, 1, 16, 32), dtype=torch.uint8), torch.zeros((2, 1, 16, 32), dtype=torch.uint8),
                     torch.zeros((2, 1, 16, 2), dtype=torch.uint8), torch.zeros((2, 1, 16, 2), dtype=torch.uint8))
    for T in (-(1 << 40), 1 << 40):
        with pytest.raises(ValueError):
            beam.attn_prompt_workspace(c, 1, T, 100, device="cpu")
    assert beam.attn_prompt_workspace(beam.AttnCfg(window=0), 1, 1, 131072, device="cpu").numel() > 256
