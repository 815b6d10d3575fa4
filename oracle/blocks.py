"""fp64 oracle of the attention layers' operators for long contexts, in numpy, written from their
definition: a cache in 8 bits, the pages' scores, their selection, attention over listed pages.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it imports nothing from the
product package.
"""
from __future__ import annotations

import numpy as np


def _table():
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7) / 8.0
    v = np.where(e == 0, f * 2.0 ** -6, (1 + f) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


E4M3 = _table()


def scale_value(e):
    """2^(e - 127), 255: NaN."""
    e = np.asarray(e)
    return np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))


def dequantise(codes, scales):
    """[pages, Hkv, page, D] uint8 codes and [pages, Hkv, page / 16] uint8 exponents as values."""
    return E4M3[codes] * np.repeat(scale_value(scales), 16, -1)[..., None]


def half_step(x):
    """Half the distance between the codes' values around x (|x| <= 448)."""
    with np.errstate(divide="ignore"):
        return 2.0 ** (np.maximum(np.floor(np.log2(np.abs(x))), -6) - 4)


def encode(x):
    """Codes of the nearest values, ties to even, |x| <= 448; not finite: NaN's."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0)
    step = 2 * half_step(a)
    v = np.round(a / step) * step  # (numpy rounds halves to even)
    code = np.searchsorted(E4M3[:127], v)
    assert np.array_equal(E4M3[code], v)
    code = np.where(fine, code, 127)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(most):
    """e of the smallest 2^(e - 127) with most <= 448 times it, 1 at least."""
    e = 1
    while most > 448 * 2.0 ** (e - 127):
        e += 1
    return e


def append(codes, scales, table, kv, fresh, tokens=None):
    """Appends fresh [T, Hkv, D], the rows kv - T .. kv - 1 of a sequence (the first `tokens` of
    them), to a cache in 8 bits, in place.  Returns {(page, head, block): ratio of the largest
    magnitude to the nearest border of the scale's choice}."""
    pages, Hkv, page, D = codes.shape
    T = len(fresh)
    row0 = kv - T
    end = row0 + (T if tokens is None else min(T, tokens))
    margins = {}
    for first in range(max(row0, 0) // 16 * 16, max(end, 0), 16):
        p, at = table[first // page], first % page
        if not 0 <= p < pages:
            continue
        new = [r for r in range(first, first + 16) if row0 <= r < end]
        old = [r for r in range(first, first + 16) if r < row0]
        for h in range(Hkv):
            y = fresh[[r - row0 for r in new], h]
            most = np.max(np.abs(np.where(np.isfinite(y), y, 0.0)), initial=0.0)
            e, was = exponent(most), int(scales[p, h, at // 16])
            margins[p, h, at // 16] = most / (448 * 2.0 ** (e - 127))
            if old:
                e = max(e, was)
            for r in old:
                if e != was:
                    codes[p, h, r % page] = encode(E4M3[codes[p, h, r % page]] * 2.0 ** (was - e))
            top = 448 if e < 247 else 0.9375 * 2.0 ** (255 - e)  # the last code whose value is less than 2^128
            z = y / scale_value(e)
            codes[p, h, [r % page for r in new]] = encode(np.where(np.isfinite(z), np.clip(z, -top, top), z))
            scales[p, h, at // 16] = e
    return margins


def mean_of(rows):
    """Mean key of a page's rows [held, D], and the mean magnitude."""
    return rows.mean(0), np.abs(rows).mean(0)


def scores(q, means):
    """q [T, G, D] of one key head, means [pages, D]: the largest product over G, [T, pages]."""
    return (q @ means.T).max(1)


def select(x, own, count, first, recent):
    """The pages a token reads, x [max_pages] its scores and own the page it lies in."""
    x = [-np.inf if np.isnan(v) else v for v in x[:own + 1]]
    must = [j for j in range(own + 1) if j < first or j > own - recent]
    rest = sorted((j for j in range(own + 1) if j not in must), key=lambda j: (-x[j], j))
    chosen = sorted((must + rest)[:count])
    return chosen + [-1] * (count - len(chosen))


def counting(entries, own):
    """The entries of a list that count: pages seen, each larger than every such one before it."""
    out = []
    for j in entries:
        if 0 <= j <= own and (not out or j > out[-1]):
            out.append(j)
    return out
