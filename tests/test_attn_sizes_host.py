"""Host-side checks of the sizes that the attention calls take: workspaces where
sinks reach as far as a sequence is long (no GPU, no kernel is launched)."""

import os

import pytest

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.skipif(not os.path.exists(beam.LIB_PATH), reason="library not built")


def decode_bytes(B, n, sinks, window, hq=48, hkv=8):
    c = beam.AttnCfg(n_heads=hq, n_kv_heads=hkv, window=window)
    return beam.lib().beam_moe_attn_decode_sinks_workspace_bytes(c.c(), sinks, B, n)


@pytest.mark.parametrize("hq,hkv", [(48, 8), (64, 1), (16, 16)])
@pytest.mark.parametrize("B", [1, 3, 64, 300, 5000])
@pytest.mark.parametrize("n", [100, 513, 1000, 4096, 131072, 1 << 30])
def test_sinks_beyond_every_token_need_what_all_tokens_need(B, n, hq, hkv):
    """A window and sinks that leave no token out are a call that sees every token."""
    every = decode_bytes(B, n, 0, 0, hq, hkv)
    for sinks in (n, n + 1, 100 * n, 1 << 30):
        sinks = min(sinks, 1 << 30)
        for window in (1, n // 2, n - 1):
            assert decode_bytes(B, n, sinks, window, hq, hkv) == every, (sinks, window)
            # no token lies between the sinks and the window
            assert decode_bytes(B, n, max(n - window, 0), window, hq, hkv) == every, window


@pytest.mark.parametrize("B", [1, 3, 64, 300])
def test_more_sinks_never_need_less(B):
    for n in (600, 1000, 5000, 131072):
        for window in (1, 64, 512):
            sizes = [decode_bytes(B, n, s, window) for s in (0, 1, 16, 100, 400, 1000, 4000, 130000, 1 << 29)]
            assert sizes == sorted(sizes), (n, window)


# ------------------------------------------------------------------ calls too large for a launch

A = 1 << 32          # never dereferenced: every call below is refused


@pytest.mark.parametrize("hq,hkv", [(256, 4), (256, 16), (256, 128), (256, 256), (64, 1)])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 1 << 22), (7, 5), (300, 300), (1 << 22, 1 << 22), (1 << 22, 1),
                                 (1 << 20, 1 << 20), (65536, 1 << 22)])
@pytest.mark.parametrize("n,window,sinks", [(1 << 30, 0, 0), (1 << 30, 1 << 20, 1 << 30), (1 << 30, 1, 1), (100, 0, 0)])
def test_most_heads_are_launched_or_refused(hq, hkv, B, T, n, window, sinks):
    """The most query heads there are, 1 to 64 to a key-value head: new tokens over a
    cache ask for a workspace that can be allocated, or are refused for their workgroups
    before they ask for one."""
    L = beam.lib()
    c = beam.AttnCfg(n_heads=hq, n_kv_heads=hkv, head_dim=256, window=window)
    size = L.beam_moe_attn_prompt_workspace_bytes
    assert size(beam.AttnCfg(n_heads=hq, n_kv_heads=hkv, head_dim=256, window=0).c(), 0, 1, 1, 131072) > 0   # a shape there is
    cache = beam.BeamMoeKvCache(A * 10, A * 20, None, None, 100, beam.BEAM_BF16)

    def call(ws, nbytes):
        return L.beam_moe_attn_prompt(c.c(), sinks, B, T, A, hq * 256, 1, cache, A * 2, 1024, A * 3, A * 3, n, A * 65536,
                                      None, ws, nbytes, None)

    need = size(c.c(), sinks, B, T, n)
    if (T * (hq // hkv) // 128 + B) * hkv >= 1 << 24:
        assert call(None, 0) == 2 and call(A * 6, 1 << 60) == 2
    elif need:               # without one it would be launched: not from here
        assert need <= 1 << 30
        assert call(None, 0) == 3 and call(A * 6, need - 1) == 3 and call(A * 6 + 4, need) == 3
