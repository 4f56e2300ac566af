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
