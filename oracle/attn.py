"""The attention sublayer's operators in plain fp64 numpy: per-head norm with
the position rotation, cache rows, attention of one new token.

[TS] "Architecture" and [VL] attention section: 48 query heads over 8
key-value heads of 128, per-head RMSNorm of queries and keys, rotary
positions in sliding-window layers, queries scaled by (1 + p/2048)^0.1 in
full-attention layers.
"""

from __future__ import annotations

import numpy as np


def norm_rope_row(x, gamma, eps, p, inv_freq, interleaved=False, factor=1.0):
    """One head row x [D]: RMSNorm (gamma None: none), rotation of its first
    2 * len(inv_freq) elements by the angles p * inv_freq, times factor."""
    x = np.asarray(x, np.float64)
    if gamma is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(gamma, np.float64)
    y = x.copy()
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a = float(p) * float(inv_freq[i])
        iu, iw = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[iu] = x[iu] * np.cos(a) - x[iw] * np.sin(a)
        y[iw] = x[iw] * np.cos(a) + x[iu] * np.sin(a)
    return y * factor


def ssmax_factor(p, length, exponent):
    """(1 + max(p, 0)/length)^exponent, 1 for length 0."""
    return 1.0 if length == 0 else (1.0 + max(float(p), 0.0) / length) ** exponent


def cached_rows(cache, page_table_row, tokens, n_pages):
    """Rows [len(tokens), h, D] of cache [n_pages, h, P, D] at a sequence's
    tokens, and which of them lie on a page of the cache."""
    P = cache.shape[2]
    rows = np.zeros((len(tokens),) + (cache.shape[1], cache.shape[3]), np.float64)
    there = np.zeros(len(tokens), bool)
    for i, t in enumerate(tokens):
        j = t // P
        page = int(page_table_row[j]) if 0 <= j < len(page_table_row) else -1
        if 0 <= page < n_pages:
            rows[i], there[i] = cache[page, :, t % P], True
    return rows, there


def decode_attention(q, k, v, scale):
    """q [h, G, D] over keys and values [n, h, D]: (out [h, G, D], lse [h, G],
    sum of probabilities times |v|); n = 0 gives 0 and -inf."""
    h, G, D = q.shape
    out, mag = np.zeros((h, G, D)), np.zeros((h, G, D))
    lse = np.full((h, G), -np.inf)
    if k.shape[0] == 0:
        return out, lse, mag
    for i in range(h):
        z = scale * (q[i] @ k[:, i].T)                 # [G, n]
        top = z.max(1, keepdims=True)
        e = np.exp(z - top)
        lse[i] = top[:, 0] + np.log(e.sum(1))
        w = e / e.sum(1, keepdims=True)
        out[i], mag[i] = w @ v[:, i], w @ np.abs(v[:, i])
    return out, lse, mag


def seen(n, length, window, sinks):
    """[n, length] truth values: the i-th of n new tokens, at p = length - n + i,
    sees the tokens j <= p with j > p - window, or j < sinks, or window 0."""
    p = length - n + np.arange(n)[:, None]
    j = np.arange(length)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks) | (window == 0))


def masked_attention(q, k, v, mask, scale):
    """q [n, h, G, D] over keys and values [L, h, D] where mask [n, L]: (out
    [n, h, G, D], lse [n, h, G], sum of probabilities times |v|); a row that
    sees nothing gives 0 and -inf."""
    n, h, G, D = q.shape
    out, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((n, h, G), -np.inf)
    some = mask.any(1)
    if not some.any():
        return out, lse, mag
    m = mask[some][:, None, :]
    for i in range(h):
        z = np.where(m, scale * (q[some, i] @ k[:, i].T), -np.inf)     # [rows, G, L]
        top = z.max(2, keepdims=True)
        e = np.exp(z - top)
        lse[some, i] = top[..., 0] + np.log(e.sum(2))
        w = e / e.sum(2, keepdims=True)
        out[some, i], mag[some, i] = w @ v[:, i], w @ np.abs(v[:, i])
    return out, lse, mag
