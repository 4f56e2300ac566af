"""Host-side tests of the attention sublayer where a wrong answer is easy to
miss (no GPU, no kernel is launched)."""

import ctypes
import os

import pytest
import torch

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.skipif(not os.path.exists(beam.LIB_PATH), reason="library not built")
DLPACK_CPU = 1


# ------------------------------------------------------------------ what the native marshalling makes of a call

ENTRIES = ("qk_norm_rope", "qk_norm_rope_cache", "kv_write", "kv_read", "attn_decode")


class Stub:
    """Entry points that note their calls and return `status`, bound for host tensors."""

    def __init__(self, status):
        from expert_routed_ffn_amd import _bind
        self.calls, self.status, self.bind = [], status, _bind
        L = beam.lib()
        self.keep = []
        for f in ENTRIES:
            types = getattr(L, "beam_moe_" + f).argtypes
            self.keep.append(ctypes.CFUNCTYPE(ctypes.c_int32, *types)(lambda *a, f=f: self.called(f, a)))
        at = [ctypes.cast(k, ctypes.c_void_p).value for k in self.keep]
        _bind.bind(torch.Tensor.__dlpack_c_exchange_api__, DLPACK_CPU, *at, beam.BeamError)

    def called(self, f, args):
        self.calls.append((f, args))
        return self.status


@pytest.fixture
def stub():
    made = []

    def make(status):
        made.append(Stub(status))
        return made[-1]
    yield make
    from expert_routed_ffn_amd import _bind
    L = beam.lib()
    at = [ctypes.cast(getattr(L, "beam_moe_" + f), ctypes.c_void_p).value for f in ENTRIES]
    _bind.bind(torch.Tensor.__dlpack_c_exchange_api__, 10, *at, beam.BeamError)   # no stub is called any more
    beam._native = None                                     # bound anew by the next call


def native_args():
    cfg = beam.AttnCfg(2, 1, 64, 0, False, 0, 16)
    x, i = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    kv = torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    cache = beam.BeamMoeKvCache(pages.data_ptr(), pages.data_ptr(), None, None, 2, beam.BEAM_BF16)
    table, off = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    return {
        "qk_norm_rope": (cfg._c, x, kv, i, x, kv, None, None, None),
        "qk_norm_rope_cache": (cfg._c, x, kv, kv, i, i, x, cache, pages, None, None, None),
        "kv_write": (cfg._c, kv, kv, i, cache, pages),
        "kv_read": (cfg._c, cache, pages, table, off, kv, kv.clone(), None),
        "attn_decode": (cfg._c, x, cache, pages, table, i, 32, x.clone(), None, None),
    }, (cfg, x, i, kv, pages)


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_that_failed_in_hip_is_made_once(stub, name):
    """A launch failure may have enqueued work, and norm and rotation may run
    in place, so the call raises; it is not handed on to be made again."""
    s, (args, keep) = stub(4), native_args()
    with pytest.raises(beam.BeamError) as e:
        getattr(s.bind, name)(*args[name])
    assert e.value.status == 4 and "beam_moe_" + name in str(e.value)
    assert [f for f, _ in s.calls] == [name]


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("status,want", [(0, True), (1, False), (2, False), (3, False)])
def test_refused_and_good_calls(stub, name, status, want):
    """Only a refusal of the arguments, which enqueues nothing, is handed on."""
    s, (args, keep) = stub(status), native_args()
    assert getattr(s.bind, name)(*args[name]) is want
    assert [f for f, _ in s.calls] == [name]


# ------------------------------------------------------------------ what a launch can hold

@pytest.mark.parametrize("N", [1, 511, 4096, (1 << 22) + 1, (1 << 24) - 1, 1 << 24, (1 << 25) + 7, 1 << 26])
def test_every_read_back_that_is_accepted_can_be_launched(N):
    """Output rows per workgroup: between one and the 64 that a wave looks up,
    and so many that a launch stays below 2^32 threads."""
    rows = beam.lib()._ZN4beam12kv_read_rowsEiii
    rows.argtypes, rows.restype = [ctypes.c_int32] * 3, ctypes.c_int32
    for hkv in (1, 2, 3, 8, 16, 32, 33, 64, 100, 256):
        for D in (64, 128, 256):
            r = rows(N, hkv, D)
            assert 1 <= r <= 64
            assert -(-N // r) * 256 < 1 << 32, (N, hkv, D, r)


# ------------------------------------------------------------------ integers beyond 32 bits

@pytest.mark.parametrize("field", ["n_heads", "n_kv_heads", "head_dim", "rope_dim", "rope_interleaved", "window",
                                   "page_size"])
@pytest.mark.parametrize("by", [1 << 32, -(1 << 32), 1 << 40])
def test_a_configuration_is_not_cut_to_32_bits(field, by):
    """Taken modulo 2^32, a window of 2^32 tokens would be none at all."""
    good = getattr(beam.AttnCfg(), field)
    assert getattr(beam.AttnCfg(**{field: good})._c, field) == good
    with pytest.raises(ValueError, match=field):
        beam.AttnCfg(**{field: int(good) + by})


@pytest.mark.parametrize("B,max_len", [(1, (1 << 32) + 100), (1, -(1 << 32)), ((1 << 32) + 1, 100)])
def test_a_workspace_is_not_cut_to_32_bits(B, max_len):
    with pytest.raises(ValueError):
        beam.attn_workspace(beam.AttnCfg(), B, max_len, device="cpu")
    assert beam.attn_workspace(beam.AttnCfg(window=0), 1, 131072, device="cpu").numel() > 256


# ------------------------------------------------------------------ parts of long sequences

@pytest.mark.parametrize("hq,hkv", [(48, 8), (8, 8), (64, 1), (32, 32)])
@pytest.mark.parametrize("B", [2, 65, 257, 300, 1000, 2047, 2048, 4095])
def test_a_long_sequence_among_many_can_be_cut(hq, hkv, B):
    """However many sequences beside it, below 4096: there is a workspace for
    parts, and it does not grow as sequences times parts."""
    L = beam.lib()
    cfg = beam.AttnCfg(n_heads=hq, n_kv_heads=hkv, window=0)
    rows = L.beam_moe_attn_workspace_bytes(cfg.c(), B, 131072) / (hq * 130 * 4)
    assert rows >= B + 31                                   # one of 131072 tokens in parts of 4096, the rest whole
    assert rows <= 4096 + 512 + B + 1
    assert L.beam_moe_attn_workspace_bytes(cfg.c(), B, 1 << 30) > 0
