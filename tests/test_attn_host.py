"""Host-side checks of the attention sublayer's entry points (no GPU, no
kernel is launched): invalid calls get the documented status before anything
is enqueued, and empty calls are no-ops."""

import ctypes
import os

import pytest
import torch

beam = pytest.importorskip("expert_routed_ffn_amd")

# never dereferenced: every call below fails validation first (or has nothing to do)
A = 1 << 32
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(beam.LIB_PATH):
        pytest.skip("library not built")
    return beam.lib()


def cfg(**kw):
    return beam.AttnCfg(**kw)


def kv(k=A * 10, v=A * 20, ks=None, vs=None, n=100, dt=beam.BEAM_BF16):
    return beam.BeamMoeKvCache(k, v, ks, vs, n, dt)


def rope(L, c=None, T=8, q=A, qs=8192, k=A + 12288, ks=8192, dt=1, gq=A * 2, gk=A * 2, pos=A * 3, fr=A * 3, qo=A * 4,
         ko=A * 5):
    return L.beam_moe_qk_norm_rope((c or cfg()).c(), T, q, qs, k, ks, dt, gq, gk, pos, fr, qo, ko, None)


def rope_cache(L, c=None, T=8, q=A, qs=8192, k=A + 12288, ks=8192, v=A + 14336, vs=8192, dt=1, gq=A * 2, gk=A * 2,
               pos=A * 3, fr=A * 3, sl=A * 3, qo=A * 4, cache=None):
    return L.beam_moe_qk_norm_rope_cache((c or cfg()).c(), T, q, qs, k, ks, v, vs, dt, gq, gk, pos, fr, sl, qo,
                                         cache if cache is not None else kv(), None)


def write(L, c=None, T=8, k=A, ks=1024, v=A * 2, vs=1024, dt=1, sl=A * 3, cache=None):
    return L.beam_moe_kv_write((c or cfg()).c(), T, k, ks, v, vs, dt, sl, cache if cache is not None else kv(), None)


def read(L, c=None, B=4, N=100, cache=None, tab=A, mp=8, off=A * 2, first=None, ko=A * 3, vo=A * 4, dt=1):
    return L.beam_moe_kv_read((c or cfg()).c(), B, N, cache if cache is not None else kv(), tab, mp, off, first, ko,
                              vo, dt, None)


def decode(L, c=None, B=4, q=A, qs=6144, dt=1, cache=None, tab=A * 2, mp=1024, lens=A * 3, ml=60000, out=A * 4,
           lse=None, ws=None, wsb=0):
    c = c or cfg(window=0)
    return L.beam_moe_attn_decode(c.c(), B, q, qs, dt, cache if cache is not None else kv(), tab, mp, lens, ml, out,
                                  lse, ws, wsb, None)


@pytest.mark.parametrize("bad,want", [
    (dict(n_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=-1), 1), (dict(head_dim=96), 2),
    (dict(head_dim=192), 2), (dict(n_heads=50), 2), (dict(n_heads=264, n_kv_heads=8), 2),
    (dict(n_heads=65, n_kv_heads=1), 2), (dict(rope_dim=-16), 1), (dict(rope_dim=144), 1), (dict(rope_dim=24), 2),
    (dict(rope_interleaved=2), 1), (dict(window=-1), 1), (dict(page_size=0), 1), (dict(page_size=8), 2),
    (dict(page_size=48), 2), (dict(page_size=2048), 2), (dict(ssmax_len=-1.0), 1), (dict(ssmax_len=float("nan")), 1),
    (dict(ssmax_exp=float("inf")), 1), (dict(softmax_scale=0.0), 1), (dict(softmax_scale=-1.0), 1),
    (dict(softmax_scale=float("inf")), 1), (dict(rms_eps=-1.0), 1), (dict(rms_eps=float("nan")), 1),
])
def test_invalid_cfg(L, bad, want):
    c = cfg(**bad)
    assert rope(L, c) == want and rope_cache(L, c) == want and write(L, c) == want
    assert read(L, c) == want and decode(L, c) == want
    assert L.beam_moe_attn_workspace_bytes(c.c(), 4, 4096) == 0


def test_null_cfg(L):
    assert L.beam_moe_kv_write(None, 8, A, 1024, A, 1024, 1, A, kv(), None) == 1


def test_nothing_to_do(L):
    c = cfg()
    assert L.beam_moe_qk_norm_rope(c.c(), 0, None, 0, None, 0, 1, None, None, None, None, None, None, None) == 0
    assert L.beam_moe_qk_norm_rope_cache(c.c(), 0, None, 0, None, 0, None, 0, 1, None, None, None, None, None, None,
                                         None, None) == 0
    assert L.beam_moe_kv_write(c.c(), 0, None, 0, None, 0, 1, None, None, None) == 0
    assert L.beam_moe_kv_read(c.c(), 0, 10, None, None, 0, None, None, None, None, 1, None) == 0
    assert L.beam_moe_kv_read(c.c(), 4, 0, None, None, 0, None, None, None, None, 1, None) == 0
    assert L.beam_moe_attn_decode(c.c(), 0, None, 0, 1, None, None, 0, None, 0, None, None, None, 0, None) == 0


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 22) + 1), dict(dt=2), dict(dt=3), dict(dt=9), dict(q=None), dict(k=None), dict(q=A + 8),
    dict(k=A + 12290), dict(qs=6136), dict(qs=6147), dict(ks=1016), dict(gq=None), dict(gk=None), dict(gq=A * 2 + 4),
    dict(pos=None), dict(pos=A * 3 + 2), dict(fr=None), dict(qo=None), dict(qo=A * 4 + 8),
    dict(qo=A),                # in place only where the rows are dense
    dict(qo=A + 16),           # overlaps q
])
def test_norm_rope_arguments(L, bad):
    assert rope(L, **bad) == 1 and rope_cache(L, **bad) == 1


def test_norm_rope_more_arguments(L):
    assert rope(L, ko=None) == 1 and rope(L, ko=A * 5 + 4) == 1
    assert rope(L, ko=A * 4 + 1024) == 1       # overlaps q_out
    assert rope(L, ko=A + 12288) == 1          # k is not dense
    assert rope_cache(L, v=None) == 1 and rope_cache(L, vs=1000) == 1
    assert rope_cache(L, sl=None) == 1 and rope_cache(L, sl=A * 3 + 1) == 1
    assert rope_cache(L, qo=A * 7, v=A * 7 + 1024, vs=1024) == 1    # q_out over v


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 4), dict(n=0), dict(n=-5), dict(dt=beam.BEAM_MXFP4),
    dict(dt=beam.BEAM_FP8_E4M3), dict(dt=beam.BEAM_FP8_E4M3, ks=A), dict(dt=beam.BEAM_FP8_E4M3, ks=A, vs=A + 4),
    dict(dt=17),
])
def test_cache_arguments(L, bad):
    c = kv(**bad)
    assert rope_cache(L, cache=c) == 1 and write(L, cache=c) == 1 and read(L, cache=c) == 1
    assert decode(L, cache=c, ws=A * 6, wsb=GB * 8) == 1


def test_cache_of_too_many_slots(L):
    c = kv(n=1 << 25)    # times 64 tokens = 2^31
    assert write(L, cache=c) == 2 and read(L, cache=c) == 2 and decode(L, cache=c) == 2


@pytest.mark.parametrize("bad", [dict(T=-1), dict(dt=2), dict(k=None), dict(v=None), dict(ks=1000), dict(vs=1028),
                                 dict(k=A + 2), dict(sl=None)])
def test_write_arguments(L, bad):
    assert write(L, **bad) == 1


@pytest.mark.parametrize("bad", [dict(B=-1), dict(N=-1), dict(N=(1 << 26) + 1), dict(mp=-1), dict(dt=2), dict(tab=None), dict(off=None),
                                 dict(off=A + 2), dict(first=A + 1), dict(ko=None), dict(vo=None), dict(ko=A * 3 + 4),
                                 dict(vo=A * 3), dict(vo=A * 3 + 2048)])
def test_read_arguments(L, bad):
    assert read(L, **bad) == 1


@pytest.mark.parametrize("bad,want", [
    (dict(B=-1), 1), (dict(B=(1 << 22) + 1), 1), (dict(mp=-1), 1), (dict(ml=-1), 1), (dict(ml=(1 << 30) + 1), 1),
    (dict(dt=2), 1), (dict(dt=0), 2), (dict(q=None), 1), (dict(qs=6140), 1), (dict(out=None), 1), (dict(out=A), 1),
    (dict(out=A * 4 + 2), 1), (dict(tab=None), 1), (dict(lens=None), 1), (dict(lens=A * 3 + 1), 1),
    (dict(lse=A + 1), 1), (dict(), 3), (dict(ws=A * 6, wsb=1024), 3), (dict(ws=A * 6 + 4, wsb=GB * 8), 3),
])
def test_decode_arguments(L, bad, want):
    assert decode(L, **bad) == want


def test_decode_dtypes(L):
    ws = dict(ws=None)
    assert decode(L, cache=kv(dt=beam.BEAM_F32), dt=1, **ws) == 2     # fp32 cache, bf16 queries
    assert decode(L, cache=kv(dt=beam.BEAM_F32), dt=0, **ws) == 3     # past the dtype check
    assert decode(L, cache=kv(dt=beam.BEAM_FP8_E4M3, ks=A, vs=A), dt=0, **ws) == 2


def test_decode_too_many_parts(L):
    assert decode(L, B=(1 << 23) // 48 + 1, ml=64, out=A * 100) == 2      # one sequence too many for 2^23 query heads
    assert decode(L, B=1, ml=1 << 30) == 3                                 # few parts however long: on to the workspace


def test_workspace_bytes(L):
    w = lambda B, n, **kw: L.beam_moe_attn_workspace_bytes(cfg(**kw).c(), B, n)
    assert w(1, 0, window=0) == 0 and w(1, 1, window=0) == 0
    assert w(1, 131072, window=0) > 0
    assert w(4096, 131072, window=0) == 0      # enough sequences to fill the chip
    assert w(1, 131072, window=512) <= w(1, 1024, window=0)
    assert w(-1, 10) == 0 and w(1, -1) == 0 and w(1, (1 << 30) + 1) == 0


def test_native_marshalling_takes_gpu_tensors_only():
    if torch.cuda.is_available():
        pytest.skip("binds the module for a machine without a GPU")
    from expert_routed_ffn_amd import _bind
    c = cfg(n_heads=2, n_kv_heads=1, head_dim=64, rope_dim=0)
    x, i = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    args = (c._c, x, x[:, :1], i, x.clone(), x[:, :1].clone(), None, None, None)
    assert _bind.qk_norm_rope(*args) is False               # not bound to a library yet
    L = beam.lib()
    at = [ctypes.cast(getattr(L, "beam_moe_" + f), ctypes.c_void_p).value
          for f in ("qk_norm_rope", "qk_norm_rope_cache", "kv_write", "kv_read", "attn_decode")]
    _bind.bind(torch.Tensor.__dlpack_c_exchange_api__, 10, *at)
    assert _bind.qk_norm_rope(*args) is False               # tensors of the CPU
    assert _bind.qk_norm_rope(*args[:8]) is False           # too few arguments
    assert _bind.kv_write(c._c, 3, None, "x", i, i) is False
    assert _bind.kv_read(c._c, c._c, x, i, i, x, x, None) is False
    assert _bind.attn_decode(c._c, x, c._c, x, i, i, -1, x, None, None) is False
    assert _bind.qk_norm_rope_cache(*([None] * 12)) is False
    with pytest.raises(TypeError):
        _bind.bind(1, 2)


def test_binding_refusals():
    c = cfg(n_heads=2, n_kv_heads=1, head_dim=64, rope_dim=0)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        beam.beam_moe_qk_norm_rope(c, x, x[:, :1], i, x.clone(), x[:, :1].clone())     # not on a GPU
    with pytest.raises(ValueError):
        beam.KVCache(torch.zeros((2, 1, 64, 64)), torch.zeros((2, 1, 64, 64)))
    m = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    dev = -1      # the CPU, as a device index
    assert beam._heads(dev, m[:, 1:3], 3, 2, 64, m.dtype, "x")[1] == 256
    assert beam._heads(dev, m[:1, 1:3], 1, 2, 64, m.dtype, "x")[1] == 128      # one row: no stride to keep
    for bad in (m[:, ::2], m.transpose(0, 1)[:3, :2], m[:, :2].float(), m[:, :3]):
        with pytest.raises(ValueError):
            beam._heads(dev, bad, 3, 2, 64, m.dtype, "x")
