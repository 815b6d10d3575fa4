"""GPU tests of the attention-layer operators at their edges: what the softmax weights' rounding
leaves of an fp32 output and of a decode step."""
import numpy as np
import pytest
import torch

from layer_checks import numbers
from oracle import attention as ref
from test_gpu_attn import BF, F32, batch, call, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


# ------------------------------------------------------------ softmax weights


@pytest.mark.parametrize("D,H,Hkv", [(128, 12, 2), (64, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("new,kv,out", [
    ([40, 70], [40, 300], F32),             # chunks, fp32 o
    ([1, 2, 1, 3], [3, 300, 64, 130], F32),  # decode, fp32 o
    ([1, 2, 1, 3], [3, 300, 64, 130], BF),   # decode, bf16 o
])
def test_weights_in_two_parts(jb, D, H, Hkv, new, kv, out):
    """Relative to sum w |v|: a weight in two bf16 parts, the first cut off (less than 2^-7 of it
    left), the second rounded by half a step: 2^-15.  A score is off by (D + 6) 2^-24 sum |q k| scale
    (a product and a sum each, the scaling, the exponent's argument), which moves weights up and
    down: twice.  Sums of at most kv terms, above and below: 2 kv 2^-24.  Exponentials and the few
    rescalings: 2^-20.  A bf16 o by half a step, 2^-8 |o|, more."""
    d = batch(new, kv, H, Hkv, D, 16, BF, seed=D + len(new))
    d["q"] = d["q"] * 0.25   # (scores whose own error is small)
    r = call(jb, d, out_dtype=out, max_seqlen=max(new))   # (at most 3 tokens: 18 rows and less, the decode form)
    numbers(r["o"])
    q, o = f64(d["q"]), f64(r["o"])
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        k, v = (ref.gather(f64(d[c]), d["table"][b].tolist(), l) for c in ("k_cache", "v_cache"))
        eo, _, mag, big = ref.attend(q[at:at + t], k, v)
        tol = mag * (2.0 ** -15 + 2 * (D + 6) * 2.0 ** -24 * big[..., None] + 2 * l * 2.0 ** -24 + 2.0 ** -20)
        if out == BF:
            tol = tol + 2.0 ** -8 * (np.abs(eo) + tol)
        far = np.abs(o[at:at + t] - eo)
        assert (far <= tol).all(), (b, (far / tol).max())
        at += t
