"""Rotary positions with several axes, the paged e4m3 cache and attention over it, fp64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

The pages have no counterpart.  Definitions:
  * rotation: pair j of axis a turns by pos_a * theta^(-j / p_a) (oracle/rope.py's
    frequencies); pair i of a row is (2i, 2i+1) or (i, i + n); elements past the
    2n rotated ones pass through; the inverse turns back;
  * append: the scale of a page that gets new tokens is 2^e, the smallest with
    448 * 2^e >= the largest magnitude among them, e >= -64 (NaN if that is not
    finite); a page that already holds tokens of the sequence keeps its old scale
    if that is larger, and its older codes become e4m3(code * old / new);
  * attention: softmax(scale q.k) v over code * scale of the page; row r of n sees
    key j of L iff j < L and (c == 0 or j < (L - n) + (r // c + 1) * c).
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode
from .rope import axis_frequencies


def rotate_axes(x, pos, pairs, theta=10000.0, half=False, inverse=False):
    """x [T, H, d], pos int [T, axes] -> rotated, fp64."""
    x = np.asarray(x, np.float64)
    pos = np.asarray(pos, np.int64).astype(np.float64)
    ang = np.concatenate([pos[:, a:a + 1] * w[None] for a, w in enumerate(axis_frequencies(pairs, theta))], 1)[:, None]
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    n = sum(pairs)
    lo, hi = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y = x.copy()
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def page_scale(amax):
    """2^e, the smallest with 448 * 2^e >= amax, e >= -64; NaN if amax is not finite."""
    if not np.isfinite(amax):
        return np.float64(np.nan)
    e = -64
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def append(x, pages, scale, table, cache_len, cu_new):
    """Appends x [N, H, d] (values, fp64 or fp32) in place: pages uint8 [P, H, page, d], scale fp64 [P, H]."""
    page = pages.shape[2]
    for b in range(table.shape[0]):
        for t in range(cu_new[b], cu_new[b + 1]):
            j = cache_len[b] + t - cu_new[b]
            if t > cu_new[b] and j % page:
                continue                                    # handled with its page's first new token
            pg, off = table[b, j // page], j % page
            n = min(page - off, cu_new[b + 1] - t)
            for h in range(pages.shape[1]):
                v = np.asarray(x[t:t + n, h], np.float64)
                need = page_scale(np.abs(v).max() if not np.isnan(v).any() else np.nan)
                old = scale[pg, h]
                new = need if off == 0 else (np.nan if np.isnan(need) or np.isnan(old) else max(old, need))
                if np.isnan(new):
                    pages[pg, h, off:off + n] = 0
                else:
                    if off and new != old:
                        was = e4m3_decode(pages[pg, h, :off])
                        # a NaN code (no append writes one) stays NaN, 0x7F
                        pages[pg, h, :off] = np.where(np.isnan(was), 0x7F, e4m3_encode(np.nan_to_num(was) * (old / new)))
                    pages[pg, h, off:off + n] = e4m3_encode(v / new)
                scale[pg, h] = new


def dense_cache(pages, scale, table, b, length):
    """Values [length, H, d] of sequence b."""
    page = pages.shape[2]
    ids = table[b, :-(-length // page)]
    v = e4m3_decode(pages[ids]) * np.asarray(scale, np.float64)[ids][:, :, None, None]
    return v.transpose(0, 2, 1, 3).reshape(-1, pages.shape[1], pages.shape[3])[:length]


def limits(n, length, causal_block):
    """Keys that each of n rows sees."""
    if causal_block == 0:
        return np.full(n, length)
    r = np.arange(n)
    return np.clip(length - n + (r // causal_block + 1) * causal_block, 0, length)


def attention(q, k, v, causal_block=0, scale=None):
    """q [n, H, d], k / v [L, Hk, d] -> (o, a, s): the output, softmax(..) |v| (the sum its terms' magnitudes make)
    and the largest sum of |q||k| terms of a row's scores (times the scale), for error bounds."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, H, d = q.shape
    g = H // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    lim = limits(n, k.shape[0], causal_block)
    o, a, s = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, H, 1))
    seen = np.arange(k.shape[0])[None] < lim[:, None]
    for h in range(H):
        x = np.where(seen, scale * (q[:, h] @ k[:, h // g].T), -np.inf)
        m = x.max(1, keepdims=True, initial=-np.inf)
        p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        z = p.sum(1, keepdims=True)
        p = p / np.where(z == 0, 1.0, z)
        o[:, h], a[:, h] = p @ v[:, h // g], p @ np.abs(v[:, h // g])
        s[:, h] = (np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(k[:, h // g]).T), 0.0)).max(1, keepdims=True, initial=0.0)
    return o, a, s
