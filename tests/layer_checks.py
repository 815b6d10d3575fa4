"""Comparisons of the attention-layer tests that no NaN passes: a comparison with NaN is false,
so `not (difference > tolerance).any()` holds for a tensor of NaN."""
import torch


def numbers(t, rows=None):
    """Asserts that a tensor (its first `rows` rows) holds no NaN."""
    t = t if rows is None else t.reshape(-1, *t.shape[-2:])[:rows]
    assert not torch.isnan(t.float()).any(), "NaN in an output"
