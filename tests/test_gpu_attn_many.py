"""GPU tests of new tokens among many sequences: one long sequence beside short
ones on both sides of the number of sequences (B * n_kv_heads of 1024) from which
on it stays in one part, and sequences whose new tokens' rows are more than one
block, which a call with many blocks does not cut.  Tolerances: the head of
test_gpu_attn_prompt.py."""

import numpy as np
import pytest
import torch

import test_gpu_attn_prompt as prompts
from parity_util import over_bound, say

beam = pytest.importorskip("expert_routed_ffn_amd")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(cfg, kind, new, lens, max_len, seed, page_rows):
    n_pages = sum(-(-max(n, 1) // page_rows) for n in lens) + 2
    c, vals = prompts.filled(cfg, n_pages, kind, seed)
    table, off = prompts.sequences(new, lens, page_rows, n_pages, seed + 1)
    q = torch.randn((int(off[-1]), cfg.n_heads, cfg.head_dim), generator=prompts.gen(seed + 2), device=DEV)
    q = q.to(prompts.act_of(kind))
    out, lse = prompts.run_prompt(cfg, q, c, table, off, lens, max_len)
    ro, rl, eo, el = prompts.prompt_ref(cfg, kind, q, *vals, table, off, lens, n_pages)
    none = np.isneginf(rl)
    got, gl = prompts.f64(out), prompts.f64(lse)
    over, lover = over_bound(got, ro, eo), over_bound(gl[~none], rl[~none], el[~none])
    say(f"  out over the bound by {over:.2e}, lse by {lover:.2e}")
    assert over <= 0 and lover <= 0
    assert np.array_equal(np.isneginf(gl), none) and (got[none] == 0).all()


@pytest.mark.parametrize("kind", prompts.KINDS)
@pytest.mark.parametrize("B", [127, 128, 129, 160])
@pytest.mark.parametrize("at", [0, 100])
def test_one_long_sequence_among_many(kind, B, at):
    say(f"one of 20001 tokens among {B} {kind}")
    cfg = beam.AttnCfg(16, 8, 64, 0, False, 0, 64, softmax_scale=0.125)
    lens = [1 + 7 * b % 40 for b in range(B)]
    lens[at] = 20001
    check(cfg, kind, [1] * B, lens, 20001, 31, 64)


@pytest.mark.parametrize("kind", prompts.KINDS)
@pytest.mark.parametrize("hq,hkv,n", [(64, 1, 3), (12, 2, 22), (48, 8, 22)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 5)])
def test_more_than_a_block_of_rows_among_many(kind, hq, hkv, n, window, sinks):
    say(f"{n} tokens of {hq}/{hkv} among many {kind}")
    cfg = beam.AttnCfg(hq, hkv, 64, 0, False, window, 16, softmax_scale=0.125, sinks=sinks)
    B = 520 // hkv                                          # blocks of many sequences fill the chip
    new = [1 + b % 2 for b in range(B)]
    lens = [new[b] + b % 30 for b in range(B)]
    new[7], lens[7], new[-1], lens[-1] = n, 5000, n, n
    check(cfg, kind, new, lens, 5000, 41, 16)
