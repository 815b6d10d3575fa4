"""GPU parity of jb_qk_norm_rope, its gradient and its cache-append form with the fp64 oracle
(oracle/attention.py), and a run of append and attention together.

Bounds, per element: y = r (x c + x' s) in fp32 with c, s one product each: some ten roundings
of terms no larger than t = r (|x w| + |x' w'|), 2^-20 t; a bf16 output adds half a step, 2^-8 |y|.
The angle is exact to 2^-24 of a turn times 2 pi, well under 2^-20.  Gradients likewise with
t = r (|h| + |h'| + |n| mean|h n|); dw, a sum of N terms in fp32, by 2^-22 times the sum of
their magnitudes (chains of at most some hundred terms, then trees)."""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_gpu_attn import BF, F32, batch, check, f64

pytestmark = pytest.mark.gpu
S = 2.0 ** -20


@pytest.fixture(scope="module")
def jb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def inputs(n, H, Hkv, D, rot, dtype, seed=0, far=262144):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    d = dict(q=r(n, H, D).to(dtype), k=r(n, Hkv, D).to(dtype), wq=(1 + 0.1 * r(D)).to(dtype),
             wk=(1 + 0.1 * r(D)).to(dtype), pos=torch.randint(0, far, (n,), generator=g, dtype=torch.int32),
             inv_freq=(1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float())
    return d, {k: v.cuda() for k, v in d.items()}


def swap(x, rot, pairs):
    """|x| + |the other member of its pair|."""
    y = np.abs(x)
    a, b = ref._pairs(rot, pairs)
    z = y.copy()
    z[..., a] += y[..., b]
    z[..., b] += y[..., a]
    return z


def near(got, want, t):
    g = f64(got).reshape(want.shape)
    tol = S * t + (2.0 ** -8 * (np.abs(want) + S * t) if got.dtype == BF else 0.0)
    bad = np.abs(g - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3].tolist(), np.abs(g - want).max())


SHAPES = [  # tokens, H, Hkv, D, rot, pairs, dtype, out dtype
    (1, 12, 2, 128, 128, False, BF, BF), (37, 12, 2, 128, 128, False, BF, F32), (130, 5, 5, 64, 32, True, F32, F32),
    (77, 3, 1, 256, 64, False, BF, BF), (19, 16, 2, 128, 16, True, BF, BF), (65, 2, 2, 64, 64, False, F32, BF),
    (33, 4, 2, 256, 256, True, F32, F32), (5, 4, 1, 64, 0, False, BF, BF), (4099, 7, 1, 64, 48, False, BF, BF),
]


@pytest.mark.parametrize("n,H,Hkv,D,rot,pairs,dtype,out", SHAPES)
@pytest.mark.parametrize("mode", ["weights", "ones", "rotation"])
def test_forward(jb, n, H, Hkv, D, rot, pairs, dtype, out, mode):
    print(f"[rope n={n} H={H}/{Hkv} D={D} rot={rot} pairs={pairs} {dtype}->{out} {mode}]", flush=True)
    d, g = inputs(n, H, Hkv, D, rot, dtype, seed=n)
    w = mode == "weights"
    norm = mode != "rotation"
    y = dict(zip("qk", jb.qk_norm_rope(g["q"], g["k"], g["pos"], g["inv_freq"], g["wq"] if w else None,
                                       g["wk"] if w else None, interleaved=pairs, normalize=norm, out_dtype=out)))
    for x in "qk":
        wx = f64(d["w" + x]) if w else None
        want = ref.norm_rope(f64(d[x]), d["pos"].numpy(), d["inv_freq"].numpy(), wx, interleaved=pairs, normalize=norm)
        v = f64(d[x])
        if norm:
            v = v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6) * (1.0 if wx is None else wx)
        near(y[x], want, swap(v, rot, pairs))


@pytest.mark.parametrize("n,H,Hkv,D,rot,pairs,dtype,out", SHAPES)
@pytest.mark.parametrize("mode", ["weights", "ones", "rotation"])
def test_backward(jb, n, H, Hkv, D, rot, pairs, dtype, out, mode):
    d, g = inputs(n, H, Hkv, D, rot, dtype, seed=n + 1)
    w, norm = mode == "weights", mode != "rotation"
    gen = torch.Generator().manual_seed(n)
    dy = {x: torch.randn(d[x].shape, generator=gen).to(out) for x in "qk"}
    r = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], dy["q"].cuda(), dy["k"].cuda(),
                                 g["wq"] if w else None, g["wk"] if w else None, interleaved=pairs, normalize=norm)
    for x in "qk":
        wx = f64(d["w" + x]) if w else None
        v, pos, fr = f64(d[x]), d["pos"].numpy(), d["inv_freq"].numpy()
        dx, dw = ref.norm_rope_backward(v, pos, fr, f64(dy[x]), wx, interleaved=pairs, normalize=norm)
        t = swap(f64(dy[x]), rot, pairs)
        if norm:
            rr = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6)
            h = t * (1.0 if wx is None else np.abs(wx))
            dots = t * np.abs(v * rr)
            t = rr * (h + np.abs(v * rr) * (h * np.abs(v * rr)).mean(-1, keepdims=True))
            assert (np.abs(f64(r["dw" + x]) - dw) <= 2.0 ** -19 * dots.sum((0, 1))).all()
        else:
            assert r["dw" + x] is None
        near(r["d" + x], dx, t)


def test_gradient_against_differences(jb):
    """dq, dk, dwq, dwk along random directions against central differences of the fp64 oracle."""
    n, H, Hkv, D, rot = 9, 3, 1, 64, 32
    d, g = inputs(n, H, Hkv, D, rot, F32, seed=2)
    gen = torch.Generator().manual_seed(3)
    dy = {x: torch.randn(d[x].shape, generator=gen) for x in "qk"}
    r = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], dy["q"].cuda(), dy["k"].cuda(), g["wq"], g["wk"])
    rng = np.random.RandomState(4)
    for x in "qk":
        f = lambda v, w: (ref.norm_rope(v, d["pos"].numpy(), d["inv_freq"].numpy(), w) * f64(dy[x])).sum()
        v, w, e = f64(d[x]), f64(d["w" + x]), 1e-5
        u, uw = rng.randn(*v.shape), rng.randn(*w.shape)
        want = (f(v + e * u, w + e * uw) - f(v - e * u, w - e * uw)) / (2 * e)
        got = (f64(r["d" + x]) * u).sum() + (f64(r["dw" + x]) * uw).sum()
        size = (np.abs(f64(r["d" + x]) * u)).sum() + np.abs(f64(r["dw" + x]) * uw).sum()
        # fp32 gradients: 2^-20 of the terms; the difference's own error is about e^2
        assert abs(got - want) <= (S + 1e-8) * size, (x, got, want)


def test_in_place_strides_and_far_positions(jb):
    """q and k as slices of one projection's output, then in place; positions up to 2^31 - 1
    and negative ones."""
    n, H, Hkv, D = 50, 6, 2, 128
    d, g = inputs(n, H, Hkv, D, D, BF, seed=6)
    d["pos"][:4] = torch.tensor([2 ** 31 - 1, -1, -2 ** 31, 10 ** 9], dtype=torch.int32)
    g["pos"] = d["pos"].cuda()
    y = jb.qk_norm_rope(g["q"], g["k"], g["pos"], g["inv_freq"], g["wq"], g["wk"])
    v = f64(d["q"])
    want = ref.norm_rope(v, d["pos"].numpy(), d["inv_freq"].numpy(), f64(d["wq"]))
    near(y[0], want, swap(v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6) * f64(d["wq"]), D, False))
    wide = torch.cat([g["q"], g["k"], g["k"]], 1)
    z = jb.qk_norm_rope(wide[:, :H], wide[:, H:H + Hkv], g["pos"], g["inv_freq"], g["wq"], g["wk"])
    assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[1])
    b = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], y[0], y[1], g["wq"], g["wk"])
    b2 = jb.qk_norm_rope_backward(wide[:, :H], wide[:, H:H + Hkv], g["pos"], g["inv_freq"], y[0], y[1], g["wq"], g["wk"])
    dq, dk = y[0].clone(), y[1].clone()
    b3 = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], dq, dk, g["wq"], g["wk"], dq=dq, dk=dk)
    for x in b:
        assert torch.equal(b[x], b2[x]) and torch.equal(b[x], b3[x]), x
    jb.qk_norm_rope(g["q"], g["k"], g["pos"], g["inv_freq"], g["wq"], g["wk"], q_out=g["q"], k_out=g["k"])
    assert torch.equal(g["q"], y[0]) and torch.equal(g["k"], y[1])
    # [B, T, H, D] is the same tokens
    d, g = inputs(n, H, Hkv, D, D, BF, seed=7)
    y = jb.qk_norm_rope(g["q"], g["k"], g["pos"], g["inv_freq"])
    z = jb.qk_norm_rope(g["q"].view(5, 10, H, D), g["k"].view(5, 10, Hkv, D), g["pos"].view(5, 10), g["inv_freq"])
    assert torch.equal(z[0].view_as(y[0]), y[0]) and torch.equal(z[1].view_as(y[1]), y[1])


def test_no_tokens(jb):
    d, g = inputs(0, 4, 2, 64, 64, BF)
    q, k = jb.qk_norm_rope(g["q"], g["k"], g["pos"], g["inv_freq"])
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    r = jb.qk_norm_rope_backward(g["q"], g["k"], g["pos"], g["inv_freq"], q, k, g["wq"], g["wk"])
    assert (r["dwq"] == 0).all() and (r["dwk"] == 0).all()


def append_inputs(new, kv, H, Hkv, D, page, dtype, seed, packed=True, behind=0):
    d = batch(new, kv, H, Hkv, D, page, dtype, seed=seed, packed=packed, behind=behind)
    g = torch.Generator().manual_seed(seed + 100)
    n = sum(new) + behind
    lead = (n,) if packed else (len(new), new[0])
    d["k"] = torch.randn(*lead, Hkv, D, generator=g).to(dtype)
    d["v"] = torch.randn(*lead, Hkv, D, generator=g).to(dtype)
    d["wq"], d["wk"] = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype), (1 + 0.1 * torch.randn(D, generator=g)).to(dtype)
    d["inv_freq"] = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    return d


def append(jb, d, **kw):
    g = {k: None if v is None else v.clone().cuda() for k, v in d.items()}
    r = jb.qk_norm_rope_paged(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["table"], g["kv"], g["inv_freq"],
                              g["wq"], g["wk"], cu_seqlens=g["cu"], **kw)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,kv,packed", [
    ([1, 3, 0, 40, 1, 70], [500, 3, 10, 55, 1, 70], True),
    ([5, 2, 3], [3, 0, 100], True),          # tokens before row 0 have no place
    ([1] * 6, [1, 16, 17, 300, 64, 63], False), ([9] * 3, [9, 200, 30], False),
])
def test_append(jb, dtype, new, kv, packed):
    """Queries as jb_qk_norm_rope's at the cache rows as positions; the caches changed in the
    new tokens' rows only, keys as jb_qk_norm_rope's, values bit for bit; a page index out of
    range is left out; rows behind the last sequence stay."""
    H, Hkv, D, page, behind = 6, 2, 64, 16, 5 if packed else 0
    d = append_inputs(new, kv, H, Hkv, D, page, dtype, seed=len(new), packed=packed, behind=behind)
    lost = None
    if kv[-1] > page:
        lost = int(d["table"][len(kv) - 1, (kv[-1] - 1) // page])
        d["table"][len(kv) - 1, (kv[-1] - 1) // page] = 10 ** 6
    qo = torch.full(d["q"].shape, 9.0, dtype=dtype, device="cuda")
    r = append(jb, d, q_out=qo)
    row = np.concatenate([np.arange(l - t, l) for t, l in zip(new, kv)])
    seq = np.concatenate([np.full(t, b) for b, t in enumerate(new)])
    n = len(row)
    pos = torch.tensor(row, dtype=torch.int32).cuda()
    y = jb.qk_norm_rope(d["q"].view(-1, H, D)[:n].cuda(), d["k"].view(-1, Hkv, D)[:n].cuda(), pos, d["inv_freq"].cuda(),
                        d["wq"].cuda(), d["wk"].cuda())
    assert torch.equal(r["q"].view(-1, H, D)[:n], y[0]) and (qo.view(-1, H, D)[n:] == 9).all()
    kc, vc = d["k_cache"].clone(), d["v_cache"].clone()
    for t in range(n):
        page_at = int(d["table"][seq[t], max(row[t], 0) // page])
        if row[t] >= 0 and page_at < kc.shape[0]:
            kc[page_at, :, row[t] % page] = y[1][t].cpu()
            vc[page_at, :, row[t] % page] = d["v"].view(-1, Hkv, D)[t]
    assert torch.equal(r["k_cache"].cpu(), kc) and torch.equal(r["v_cache"].cpu(), vc)
    if lost is not None:
        assert torch.equal(r["k_cache"][lost].cpu(), d["k_cache"][lost])


def test_append_positions_of_their_own(jb):
    new, kv = [4, 1], [20, 33]
    d = append_inputs(new, kv, 4, 2, 64, 16, BF, seed=21)
    pos = torch.tensor([7, 100000, 0, 3, 5], dtype=torch.int32).cuda()
    r = append(jb, d, positions=pos)
    y = jb.qk_norm_rope(d["q"].cuda(), d["k"].cuda(), pos, d["inv_freq"].cuda(), d["wq"].cuda(), d["wk"].cuda())
    assert torch.equal(r["q"], y[0])
    assert torch.equal(r["k_cache"][int(d["table"][1, 2]), :, 0], y[1][4])


def test_malformed_offsets_stay_in_bounds(jb):
    print("[append: malformed cu_seqlens, kv_lens]", flush=True)
    d = append_inputs([20, 20, 20], [50, 50, 50], 4, 2, 64, 16, BF, seed=22)
    d["cu"] = torch.tensor([0, 900, -7, 60], dtype=torch.int32)
    d["kv"] = torch.tensor([10 ** 9, -3, 50], dtype=torch.int32)
    P = d["k_cache"].shape[0]
    guard = torch.full((P + 4, 2, 16, 64), 3.0, dtype=BF, device="cuda")
    q = torch.full((100, 4, 64), 3.0, dtype=BF, device="cuda")
    g = {k: v.cuda() for k, v in d.items()}
    jb.qk_norm_rope_paged(g["q"], g["k"], g["v"], guard[2:2 + P], g["v_cache"], g["table"], g["kv"], g["inv_freq"],
                          cu_seqlens=g["cu"], q_out=q[20:80])
    torch.cuda.synchronize()
    assert (guard[:2] == 3).all() and (guard[-2:] == 3).all() and (q[:20] == 3).all() and (q[80:] == 3).all()


def test_layer_in_serving(jb):
    """Append and attention together, as a layer runs them: a prompt in chunks and two decode
    steps of three requests in packed batches, against the oracle on whole sequences."""
    H, Hkv, D, page, window = 6, 2, 64, 16, 40
    steps = [[50, 7, 1], [33, 0, 20], [1, 1, 1], [1, 1, 1]]
    total = np.sum(steps, 0)
    g = torch.Generator().manual_seed(30)
    q, k, v = ([torch.randn(t, h, D, generator=g).to(BF) for t in total] for h in (H, Hkv, Hkv))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(BF)
    fr = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    pool = sum(-(-t // page) for t in total)
    order = iter(torch.randperm(pool, generator=g).tolist())
    table = torch.full((3, 6), -1, dtype=torch.int32)
    for b, t in enumerate(total):
        for x in range(-(-t // page)):
            table[b, x] = next(order)
    caches = [torch.full((pool, Hkv, page, D), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
    have = [0, 0, 0]
    outs, qs = [[], [], []], [[], [], []]
    for new in steps:
        pick = lambda x: torch.cat([x[b][have[b]:have[b] + t] for b, t in enumerate(new)]).cuda()
        args = pick(q), pick(k), pick(v)
        have = [h + t for h, t in zip(have, new)]
        kv = torch.tensor(have, dtype=torch.int32).cuda()
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        r = jb.qk_norm_rope_paged(*args, *caches, table.cuda(), kv, fr.cuda(), w.cuda(), w.cuda(), cu_seqlens=cu)
        a = jb.attn_paged(r["q"], *caches, table.cuda(), kv, cu_seqlens=cu, max_seqlen=max(new), window=window,
                          want_lse=True)
        for b, (i, j) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
            outs[b].append((a["o"][i:j], a["lse"][i:j]))
            qs[b].append(r["q"][i:j])
    d = dict(q=torch.cat([torch.cat(x) for x in qs]).cpu(), k_cache=torch.nan_to_num(caches[0]).cpu(),
             v_cache=torch.nan_to_num(caches[1]).cpu(), table=table)
    r = dict(o=torch.cat([x[0] for y in outs for x in y]), lse=torch.cat([x[1] for y in outs for x in y]))
    check(d, r, total.tolist(), total.tolist(), window)
    # the rotated keys in the pages are the oracle's
    for b in range(3):
        got = ref.gather(f64(caches[0]), table[b].tolist(), int(total[b]))
        x = f64(k[b])
        want = ref.norm_rope(x, np.arange(total[b]), fr.numpy(), f64(w))
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()


def test_captured_step(jb):
    """Append and decode attention in one graph, replayed while the lengths grow in place."""
    d = append_inputs([1, 1], [40, 65], 4, 2, 64, 16, BF, seed=31, packed=False)
    d["table"] = torch.cat([d["table"], torch.tensor([[-1], [-1]], dtype=torch.int32)], 1)
    g = {k: v.cuda() for k, v in d.items() if v is not None}

    def step(kc, vc):
        r = jb.qk_norm_rope_paged(g["q"], g["k"], g["v"], kc, vc, g["table"], g["kv"], g["inv_freq"], g["wq"], g["wk"])
        return jb.attn_paged(r["q"], kc, vc, g["table"], g["kv"])["o"]
    kc, vc = g["k_cache"].clone(), g["v_cache"].clone()
    step(kc, vc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(g["k_cache"], g["v_cache"])
    for i in range(5):
        g["q"].normal_()
        g["k"].normal_()
        g["v"].normal_()
        e = step(kc, vc)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, e) and torch.equal(kc, g["k_cache"]) and torch.equal(vc, g["v_cache"]), i
        g["kv"].add_(1)
