"""Pins of the attention oracle (oracle/attn.py) against torch's complex
product, softmax and attention in fp64 on the CPU, and against properties."""

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_complex_product(inter):
    g = np.random.default_rng(1)
    x, f = g.standard_normal(64), 10000.0 ** (-np.arange(0, 32, 2) / 32)
    y = oracle.norm_rope_row(x, None, 0.0, 777, f, inter)
    pairs = x[:32].reshape(16, 2) if inter else x[:32].reshape(2, 16).T
    z = torch.view_as_complex(torch.tensor(pairs.copy())) * torch.polar(torch.ones(16, dtype=torch.float64),
                                                                        torch.tensor(777 * f))
    z = torch.view_as_real(z).numpy()
    assert np.allclose(y[:32], z.reshape(-1) if inter else z.T.reshape(-1), rtol=0, atol=1e-12)
    assert np.array_equal(y[32:], x[32:])


def test_rotation_keeps_relative_positions_and_norms():
    g = np.random.default_rng(2)
    q, k, f = g.standard_normal(128), g.standard_normal(128), 10000.0 ** (-np.arange(0, 128, 2) / 128)
    at = lambda x, p: oracle.norm_rope_row(x, None, 0.0, p, f)
    assert np.isclose(at(q, 100) @ at(k, 93), at(q, 507) @ at(k, 500), rtol=0, atol=1e-9)
    assert np.isclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q))


def test_norm_matches_torch():
    g = np.random.default_rng(3)
    x, gamma = g.standard_normal(128), g.standard_normal(128)
    ref = torch.nn.functional.rms_norm(torch.tensor(x), (128,), torch.tensor(gamma), eps=1e-6).numpy()
    assert np.allclose(oracle.norm_rope_row(x, gamma, 1e-6, 5, None), ref, rtol=1e-12)
    assert oracle.ssmax_factor(2048, 2048.0, 0.1) == 2.0 ** 0.1 and oracle.ssmax_factor(-3, 2048.0, 0.1) == 1.0


def test_attention_matches_torch():
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((2, 3, 16)), g.standard_normal((40, 2, 16)), g.standard_normal((40, 2, 16))
    out, lse, _ = oracle.decode_attention(q, k, v, 0.25)
    tk, tv = torch.tensor(k).transpose(0, 1), torch.tensor(v).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q), tk, tv, scale=0.25).numpy()
    z = 0.25 * torch.tensor(q) @ tk.transpose(1, 2)
    assert np.allclose(out, ref, atol=1e-12) and np.allclose(lse, torch.logsumexp(z, -1).numpy(), atol=1e-12)
    out, lse, _ = oracle.decode_attention(q, k[:0], v[:0], 0.25)
    assert not out.any() and np.isneginf(lse).all()


def test_cached_rows_follow_the_table():
    cache = np.arange(3 * 2 * 16 * 4, dtype=np.float64).reshape(3, 2, 16, 4)
    rows, there = oracle.cached_rows(cache, [2, -1, 0], [0, 17, 35, 48], 3)
    assert list(there) == [True, False, True, False]
    assert np.array_equal(rows[0], cache[2, :, 0]) and np.array_equal(rows[2], cache[0, :, 3])
    assert not rows[1].any() and not rows[3].any()


@pytest.mark.parametrize("n,length,window,sinks", [(5, 5, 0, 0), (4, 20, 6, 0), (9, 30, 5, 3), (30, 30, 7, 2),
                                                   (3, 2, 0, 0), (1, 40, 8, 100)])
def test_masked_attention_is_one_query_at_a_time(n, length, window, sinks):
    g = np.random.default_rng(n * 100 + length)
    q, k, v = g.standard_normal((n, 2, 3, 16)), g.standard_normal((length, 2, 16)), g.standard_normal((length, 2, 16))
    mask = oracle.seen(n, length, window, sinks)
    out, lse, mag = oracle.masked_attention(q, k, v, mask, 0.25)
    for i in range(n):
        p = length - n + i
        j = [t for t in range(p + 1) if not window or p - t < window or t < sinks]
        assert list(np.nonzero(mask[i])[0]) == j
        o, l, a = oracle.decode_attention(q[i], k[j], v[j], 0.25)
        assert np.allclose(out[i], o, atol=1e-13) and np.allclose(lse[i], l) and np.allclose(mag[i], a, atol=1e-13)


def test_masked_attention_against_torch():
    g = np.random.default_rng(3)
    q, k, v = (g.standard_normal((1, 12, 32)) for _ in range(3))
    mask = oracle.seen(12, 12, 5, 2)
    want = torch.nn.functional.scaled_dot_product_attention(*(torch.tensor(x) for x in (q, k, v)),
                                                            attn_mask=torch.tensor(mask), scale=0.3)[0].numpy()
    out, _, _ = oracle.masked_attention(q[0][:, None, None], k[0][:, None], v[0][:, None], mask, 0.3)
    assert np.allclose(out[:, 0, 0], want, atol=1e-13)
