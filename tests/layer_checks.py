"""Comparisons of the attention-layer tests that no NaN passes: a comparison with NaN is false,
so `not (difference > tolerance).any()` holds for a tensor of NaN."""
import numpy as np
import torch


def numbers(t, rows=None):
    """Asserts that a tensor (its first `rows` rows) holds no NaN."""
    t = t if rows is None else t.reshape(-1, *t.shape[-2:])[:rows]
    assert not torch.isnan(t.float()).any(), "NaN in an output"


def same_kind(got, want):
    """Asserts NaN, +inf and -inf exactly where `want` has them; returns got as an array."""
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    for f in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(f(got), f(want)), (f.__name__, np.argwhere(f(got) != f(want))[:4].tolist())
    return got
