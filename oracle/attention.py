"""fp64 oracle of the attention-layer operators, in numpy, written from their definition.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it imports nothing from the
product package.  Inputs are float arrays holding the exact values given to the GPU.
"""
from __future__ import annotations

import numpy as np


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, positions, inv_freq, interleaved=False, sign=1.0):
    """x [tokens, heads, D]: pair (a, b) to (a cos - b sin, b cos + a sin)."""
    x = np.array(x, np.float64)
    a, b = _pairs(2 * len(inv_freq), interleaved)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    c, s = np.cos(t)[:, None, :], sign * np.sin(t)[:, None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, positions, inv_freq, w=None, eps=1e-6, interleaved=False, normalize=True):
    x = np.array(x, np.float64)
    if normalize:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            x = x * np.asarray(w, np.float64)
    return rotate(x, positions, inv_freq, interleaved)


def norm_rope_backward(x, positions, inv_freq, dy, w=None, eps=1e-6, interleaved=False, normalize=True):
    """(dx, dw) of norm_rope; dw sums over tokens and heads."""
    x = np.array(x, np.float64)
    g = rotate(dy, positions, inv_freq, interleaved, -1.0)
    if not normalize:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dw = (g * n).sum((0, 1))
    h = g if w is None else g * np.asarray(w, np.float64)
    return r * (h - n * (h * n).mean(-1, keepdims=True)), dw


def gather(cache, table, kv):
    """Rows 0 .. kv - 1 of one sequence: cache [pages, Hkv, page, D] -> [kv, Hkv, D]; a page
    index out of range gives rows of zeros."""
    pages, Hkv, page, D = cache.shape
    out = np.zeros((kv, Hkv, D))
    for j0 in range(0, kv, page):
        p = table[j0 // page]
        n = min(page, kv - j0)
        if 0 <= p < pages:
            out[j0:j0 + n] = np.asarray(cache[p, :, :n], np.float64).transpose(1, 0, 2)
    return out


def attend(q, k, v, window=0, scale=None):
    """One sequence: q [T, H, D], its cache rows k, v [kv, Hkv, D], the last T of them the new
    tokens'.  Returns o [T, H, D], lse [T, H], and for error bounds: the sum of weights times
    |v| [T, H, D] and the largest sum of |q_d k_d| times scale [T, H]."""
    T, H, D = q.shape
    kv, Hkv, _ = k.shape
    scale = D ** -0.5 if scale is None else scale
    q = np.asarray(q, np.float64)
    o, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, big = np.full((T, H), -np.inf), np.zeros((T, H))
    for i in range(T):
        p = kv - T + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(H):
            ks, vs = k[lo:p + 1, h * Hkv // H], v[lo:p + 1, h * Hkv // H]
            x = ks @ q[i, h] * scale
            m = x.max()
            w = np.exp(x - m)
            lse[i, h] = m + np.log(w.sum())
            w /= w.sum()
            o[i, h] = w @ vs
            mag[i, h] = w @ np.abs(vs)
            big[i, h] = (np.abs(ks) @ np.abs(q[i, h])).max() * scale
    return o, lse, mag, big
