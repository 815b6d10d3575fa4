"""GPU tests of the attention-layer operators at their edges: what the softmax weights' rounding
leaves of an fp32 output and of a decode step, values that are not finite next to the rotation."""
import numpy as np
import pytest
import torch

from layer_checks import numbers, same_kind
from oracle import attention as ref
from test_gpu_attn import BF, F32, batch, call, f64
from test_gpu_rope import inputs

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


# ------------------------------------------------- values that are not finite

BAD = [float("inf"), -float("inf"), float("nan")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("bad", BAD)
def test_unrotated_values_pass_through(jb, dtype, pairs, rot, bad):
    """The rotation does not reach past the first rot values: without the norm the rest leave as they
    came, whatever they are, and none of them is felt elsewhere; with the norm as the oracle has it."""
    n, H, Hkv, D = 5, 3, 1, 64
    d, g = inputs(n, H, Hkv, D, rot, dtype, seed=rot + 1)
    run = lambda x, **a: dict(zip("qk", jb.qk_norm_rope(x["q"], x["k"], x["pos"], x["inv_freq"], interleaved=pairs, **a)))
    clean = run(g, normalize=False)
    where = [(0, 0, rot), (1, 0, D - 1), (2, 0, 45), (4, 0, 50)]
    for x in "qk":
        for at in where:
            d[x][at] = bad
        g[x] = d[x].cuda()
    y = run(g, normalize=False)
    for x in "qk":
        for at in where:
            want = torch.tensor(bad).to(y[x].dtype)
            assert torch.equal(torch.nan_to_num(y[x][at].cpu(), 7, 8, 9), torch.nan_to_num(want, 7, 8, 9)), (x, at)
            y[x][at], clean[x][at] = 0, 0
        assert torch.equal(y[x], clean[x])
    y = run(g, wq=g["wq"], wk=g["wk"])
    for x in "qk":
        with np.errstate(invalid="ignore"):
            want = ref.norm_rope(f64(d[x]), d["pos"].numpy(), d["inv_freq"].numpy(), f64(d["w" + x]), interleaved=pairs)
        got = same_kind(y[x], want)
        fine = np.isfinite(want)
        assert (np.abs(got - want)[fine] <= 2.0 ** -7 * np.abs(want[fine]) + 1e-5).all()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("bad", BAD)
def test_unrotated_gradients_pass_through(jb, pairs, rot, bad):
    """The same of the gradient: an incoming value that is not finite and not rotated."""
    n, H, Hkv, D = 4, 2, 1, 64
    d, g = inputs(n, H, Hkv, D, rot, F32, seed=rot + 2)
    gen = torch.Generator().manual_seed(rot)
    dy = {x: torch.randn(d[x].shape, generator=gen) for x in "qk"}
    run = lambda **a: jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], dy["q"].cuda(), dy["k"].cuda(),
                                               interleaved=pairs, **a)
    clean, clean_norm = run(normalize=False), run(wq=g["wq"], wk=g["wk"])
    where = [(0, 0, rot), (2, 0, 51)]
    for x in "qk":
        for at in where:
            dy[x][at] = bad
    r, rn = run(normalize=False), run(wq=g["wq"], wk=g["wk"])
    for x in "qk":
        for at in where:
            assert torch.equal(torch.nan_to_num(r["d" + x][at].cpu(), 7, 8, 9), torch.nan_to_num(torch.tensor(bad), 7, 8, 9))
            r["d" + x][at] = clean["d" + x][at] = 0
        assert torch.equal(r["d" + x], clean["d" + x])
        with np.errstate(invalid="ignore"):
            dx, dw = ref.norm_rope_backward(f64(d[x]), d["pos"].numpy(), d["inv_freq"].numpy(), f64(dy[x]), f64(d["w" + x]),
                                            interleaved=pairs)
        same_kind(rn["d" + x], dx)
        same_kind(rn["dw" + x], dw)
        keep = torch.ones(D, dtype=torch.bool)
        keep[[at[2] for at in where]] = False
        assert torch.equal(rn["dw" + x].cpu()[keep], clean_norm["dw" + x].cpu()[keep])
