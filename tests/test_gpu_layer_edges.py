"""GPU tests of the attention-layer operators at their edges: what the softmax weights' rounding
leaves of an fp32 output and of a decode step, values that are not finite next to the rotation,
packed sequences longer than the planned length, padded batches, long sums of weight gradients."""
import numpy as np
import pytest
import torch

from layer_checks import numbers, same_kind
from oracle import attention as ref
from test_gpu_attn import BF, F32, batch, call, f64
from test_gpu_rope import append, append_inputs, inputs, swap

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


# ------------------------------------- sequences longer than the planned length


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,kv,most,window", [
    ([90, 20, 70], [200, 64, 50], 60, 0), ([90, 20], [200, 64], 60, 40), ([9, 1, 2], [300, 9, 1], 4, 0),
    ([9, 1, 2], [300, 9, 70], 4, 33),
])
def test_tokens_of_a_cut_sequence_keep_their_rows(jb, dtype, new, kv, most, window):
    """Of a sequence longer than max_seqlen the first tokens are computed: as tokens of that sequence,
    at the rows they have in it (the last one is row kv - 1), in attention and in the append."""
    H, Hkv, D, page = 6, 2, 64, 16
    d = append_inputs(new, kv, H, Hkv, D, page, dtype, seed=40 + most)
    whole, cut = append(jb, d), append(jb, d, max_seqlen=most)
    attended = {k: d[k] for k in ("q", "k_cache", "v_cache", "table", "kv", "cu")}
    o, part = call(jb, attended, window=window), call(jb, attended, window=window, max_seqlen=most)
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        here = slice(at, at + min(t, most))
        assert torch.equal(cut["q"][here], whole["q"][here]), b
        seen = f64(o["lse"][here])
        # perhaps by another kernel, its sums in another order.  lse: either is off by some 66 2^-24 sum |q k| / 8
        # and 2^-17; o: by half a step of a weight and of o itself (fp32: twice lse's error), relative to |v|
        got, some = f64(part["lse"][here]), np.isfinite(seen)
        assert np.array_equal(np.isneginf(seen), np.isneginf(got))
        assert (np.abs(got[some] - seen[some]) <= 2.0 ** -13 * (1 + np.abs(seen[some]))).all(), b
        v = np.abs(ref.gather(f64(d["v_cache"]), d["table"][b].tolist(), l)).max() if l else 0.0
        assert (np.abs(f64(part["o"][here]) - f64(o["o"][here])) <= (1.1 * 2.0 ** -6 if dtype == BF else 2.0 ** -14) * v).all(), b
        for i in range(t):
            row = l - t + i
            if row < 0:
                continue
            p, x = int(d["table"][b, row // page]), row % page
            src = whole if i < most else d
            for c in ("k_cache", "v_cache"):
                assert torch.equal(cut[c][p, :, x].cpu(), src[c][p, :, x].cpu()), (b, i)
        at += t


# --------------------------------------------------------------- padded batches


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("behind", [1, 60])
def test_padded_decode_batch(jb, dtype, behind):
    """Single tokens, packed, with rows behind them that nobody owns (a batch padded to a size of its
    own): their outputs stay, the others are as without them."""
    new, kv = [1, 1, 0, 1], [90, 300, 5, 17]
    d = append_inputs(new, kv, 4, 2, 64, 16, dtype, seed=50, behind=behind)
    bare = dict(d, **{x: d[x][:3] for x in "qkv"})
    qo = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
    r, e = append(jb, d, max_seqlen=1, q_out=qo), append(jb, bare, max_seqlen=1)
    assert torch.equal(r["q"][:3], e["q"]) and (qo[3:] == 5).all()
    for c in ("k_cache", "v_cache"):
        assert torch.equal(r[c], e[c])
    attended = {k: d[k] for k in ("q", "k_cache", "v_cache", "table", "kv", "cu")}
    o = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
    r, e = call(jb, attended, max_seqlen=1, o=o), call(jb, dict(attended, q=bare["q"]), max_seqlen=1)
    numbers(r["o"])
    assert (o[3:] == 5).all()
    # (perhaps by another kernel: half a step of a weight and of o, each side; fp32 as above)
    far = (r["o"][:3].float() - e["o"].float()).abs().max()
    assert far <= (1.1 * 2.0 ** -6 if dtype == BF else 2.0 ** -14) * d["v_cache"].float().abs().max()


# ---------------------------------------------------------- weight gradients


@pytest.mark.parametrize("n,H,Hkv,adds", [(1, 1, 1, 1), (2, 3, 1, 6), (65536, 2, 1, 94)])
def test_sums_of_the_weights_gradients(jb, n, H, Hkv, adds):
    """dwq, dwk relative to the sum of |n| (|y| + |y'|).  A term, in units of 2^-24: cosine and sine off
    by 5 (the fraction of a turn rounded, 1.6; the series and its roundings), two roundings of
    y c + y' s; of n = x r 11 (8 + 5 of the sum of squares, halved by the root, eps, the root 2, the
    quotient, the product): 18.  And one for each sum on the longest way: all terms at most; for
    many tokens a lane's 3 x 2, 32 groups of a workgroup, 24 workgroups of a thread and 32 threads."""
    D = 64
    d, g = inputs(n, H, Hkv, D, D, F32, seed=n)
    gen = torch.Generator().manual_seed(n + 1)
    dy = {x: torch.randn(d[x].shape, generator=gen) for x in "qk"}
    r = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], dy["q"].cuda(), dy["k"].cuda(), g["wq"], g["wk"])
    for x in "qk":
        v = f64(d[x])
        _, dw = ref.norm_rope_backward(v, d["pos"].numpy(), d["inv_freq"].numpy(), f64(dy[x]), f64(d["w" + x]))
        size = (swap(f64(dy[x]), D, False) * np.abs(v) / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6)).sum((0, 1))
        assert (np.abs(f64(r["dw" + x]) - dw) <= (18 + adds) * 2.0 ** -24 * size).all(), x
