"""CPU tests around the attention-layer operators: the comparisons of their GPU tests and the
binding's and the library's handling of calls at their limits."""
import numpy as np
import pytest
import torch

from oracle import attention as ref


def test_comparisons_refuse_nan():
    """An output of NaN passes neither comparison of the strict run of the GPU tests; the right one
    passes both."""
    import test_gpu_attn
    import test_gpu_rope
    from test_gpu_layer_strict import strict
    check, near = strict(test_gpu_attn.check, test_gpu_rope.near)
    new, kv, H, Hkv, D, page = [3, 1], [20, 7], 2, 1, 64, 16
    d = test_gpu_attn.batch(new, kv, H, Hkv, D, page, torch.float32)
    o, lse = [], []
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        k, v = (ref.gather(d[c].numpy().astype(np.float64), d["table"][b].tolist(), l) for c in ("k_cache", "v_cache"))
        eo, el, _, _ = ref.attend(d["q"][at:at + t].numpy(), k, v)
        o.append(eo), lse.append(el)
        at += t
    o, lse = (torch.tensor(np.concatenate(x), dtype=torch.float32) for x in (o, lse))
    check(d, dict(o=o, lse=lse), new, kv)
    for name, i in (("o", (0, 1, 5)), ("o", (3, 0, 63)), ("lse", (2, 1))):
        r = dict(o=o.clone(), lse=lse.clone())
        r[name][i] = float("nan")
        with pytest.raises(AssertionError):
            check(d, r, new, kv)
    # rows behind the last sequence are nobody's
    r = dict(o=torch.cat([o, o[:1] * float("nan")]), lse=torch.cat([lse, lse[:1] * float("nan")]))
    check(dict(d, q=torch.cat([d["q"], d["q"][:1]])), r, new, kv)
    want = np.ones((2, 3, 4))
    near(torch.ones(2, 3, 4), want, want)
    for bad in (torch.full((2, 3, 4), float("nan")), torch.tensor([1.0] * 23 + [float("nan")]).view(2, 3, 4)):
        with pytest.raises(AssertionError):
            near(bad, want, want)
