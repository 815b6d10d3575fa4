"""GPU parity of attention over selected pages (jb_block_scores, jb_block_select, jb_attn_blocks) with
the fp64 oracles (oracle/blocks.py, oracle/attention.py), over caches in 16, 32 and 8 bits.

Bounds.  A mean is an fp32 sum of `held` rows and a division: off by at most (held + 1) 2^-24 of the
mean magnitude.  A score is an fp32 sum of exact products (bf16 queries) or of D rounded ones:
(D + 2) 2^-24 sum |q_d m_d|, with bf16 queries three sums in one (3 D + 2).  The selection is exact.
The attention's bounds are test_gpu_attn's over the listed rows."""
import numpy as np
import pytest
import torch

from layer_checks import same_kind
from oracle import attention as ref
from oracle import blocks as ref8
from test_gpu_attn import BF, F32, batch, f64
from test_gpu_attn8 import E4M3, E8M0, batch8, codes_of, jb, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

LENGTHS = {
    "edges": ([1, 2, 5, 31, 33, 64, 65], [1, 64, 65, 31, 127, 128, 300]),
    "empty rows": ([4, 3, 0, 1, 70, 1], [2, 0, 9, 0, 40, 5]),
}
CACHES = [(BF, 16), (BF, 8), (F32, 32), (F32, 8)]


def inputs(new, kv, H, Hkv, D, page, dtype, bits, seed=0, **kw):
    """(d, g): the batch with the values its caches hold, on the CPU, and as it is on the GPU."""
    if bits == 8:
        d, d8 = batch8(new, kv, H, Hkv, D, page, dtype, seed=seed, **kw)
    else:
        d = batch(new, kv, H, Hkv, D, page, dtype, seed=seed, **kw)
        d8 = dict(d, k_scales=None, v_scales=None)
    return d, on_gpu(d8)


def places(new, kv, tokens=None):
    """(token, sequence, cache row) of every token taken."""
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        for i in range(t if tokens is None else min(t, tokens)):
            yield at + i, b, l - t + i
        at += t


# ------------------------------------------------------------------ scores


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("D,H,Hkv,page", [(128, 12, 2, 64), (64, 5, 5, 16), (256, 8, 2, 32)])
@pytest.mark.parametrize("dtype,bits", CACHES)
def test_scores(jb, lengths, dtype, bits, D, H, Hkv, page):
    new, kv = LENGTHS[lengths]
    print(f"[scores {lengths} {dtype} {bits} D={D} H={H}/{Hkv} page={page}]", flush=True)
    d, g = inputs(new, kv, H, Hkv, D, page, dtype, bits, seed=D + H, behind=3)
    P, G, width = len(d["k_cache"]), H // Hkv, d["table"].shape[1]
    before = torch.randn(P, Hkv, D, generator=torch.Generator().manual_seed(1))
    out = torch.full((sum(new) + 3, Hkv, width), 5.0, device="cuda")
    means = before.cuda()
    r = jb.block_scores(g["q"], g["k_cache"], means, g["table"], g["kv"], k_scales=g["k_scales"], cu_seqlens=g["cu"],
                        scores=out)
    torch.cuda.synchronize()
    k, q = f64(d["k_cache"]), f64(d["q"])
    want, tol = f64(before), np.zeros((P, Hkv, D))
    for b, (t, l) in enumerate(zip(new, kv)):
        for j in range(max(0, l - t) // page, -(-l // page) if t else 0):
            p, held = int(d["table"][b, j]), min(page, l - j * page)
            want[p], mag = ref8.mean_of(k[p, :, :held].swapaxes(0, 1))
            tol[p] = (held + 1) * 2.0 ** -24 * mag
    got_m = same_kind(means, want)
    assert (np.abs(got_m - want) <= tol).all()
    scores = np.full((sum(new) + 3, Hkv, width), 5.0)
    slack = np.zeros_like(scores)
    scores[:sum(new)] = -np.inf
    for t, b, p in places(new, kv):
        for h in range(Hkv):
            for j in range(p // page + 1):
                m = got_m[int(d["table"][b, j]), h]
                qs = q[t, h * G:(h + 1) * G]
                scores[t, h, j] = (qs @ m).max()
                slack[t, h, j] = (3 * D + 2) * 2.0 ** -24 * (np.abs(qs) @ np.abs(m)).max()
    got = same_kind(r["scores"], scores)
    fine = np.isfinite(scores)
    assert (np.abs(got[fine] - scores[fine]) <= slack[fine]).all()


def test_scores_of_a_dense_batch(jb):
    """[B, T, H, D] and [B, H, D]; more pages than a workgroup takes; means only; a page out of range
    scores as zeros and is not written."""
    for T, H, Hkv in ((1, 12, 2), (40, 4, 4)):
        kv = [40, 3000, 700]
        d, g = inputs([T] * 3, kv, H, Hkv, 64, 16, BF, 16, seed=2, packed=False)
        d["table"][1, 5] = -1
        g["table"] = d["table"].cuda()
        k, q = f64(d["k_cache"]), f64(d["q"])
        means = np.stack([k[p].mean(1) for p in range(len(k))])
        m = torch.from_numpy(means).float().cuda()
        args = (g["k_cache"], m, g["table"], g["kv"])
        if T == 1:
            g["q"] = g["q"][:, 0]
        r = jb.block_scores(g["q"], *args)
        assert r["scores"].shape == (*g["q"].shape[:-2], Hkv, d["table"].shape[1])
        got_m, got = f64(m), f64(r["scores"]).reshape(3, T, Hkv, -1)
        for b, l in enumerate(kv):
            for i in range(T):
                own = (l - T + i) // 16
                for h in range(Hkv):
                    qs = q[b, i, h * (H // Hkv):(h + 1) * (H // Hkv)]
                    ms = np.stack([got_m[p, h] if 0 <= p < len(k) else np.zeros(64) for p in d["table"][b, :own + 1].tolist()])
                    slack = 194 * 2.0 ** -24 * (np.abs(qs) @ np.abs(ms).T).max(0)
                    assert (np.abs(got[b, i, h, :own + 1] - (qs @ ms.T).max(0)) <= slack).all()
                    assert (got[b, i, h, own + 1:] == -np.inf).all()
        again = torch.from_numpy(means).float().cuda()
        r2 = jb.block_scores(g["q"], g["k_cache"], again, g["table"], g["kv"], want_scores=False)
        assert r2["scores"] is None and torch.equal(again, m)


def test_scores_that_are_not_numbers(jb):
    """A NaN of any query head of the group stays; means of pages that are not seen have no part."""
    d, g = inputs([2], [70], 6, 2, 64, 16, BF, 16, seed=3)
    g["q"][0, 1, 7] = float("nan")
    g["q"][1, 4, 9] = float("inf")
    means = torch.full((len(d["k_cache"]), 2, 64), float("nan"), device="cuda")
    means[g["table"][0].long()] = 1.0
    x = jb.block_scores(g["q"], g["k_cache"], means, g["table"], g["kv"], cu_seqlens=g["cu"])["scores"]
    assert torch.isnan(x[0, 0]).all() and torch.isfinite(x[0, 1]).all() and torch.isfinite(x[1, 0]).all()
    assert not torch.isfinite(x[1, 1]).any()


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [40, 3000, 700]), ([40, 33, 5], [40, 3000, 700])])
@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF, 64, 4, 2), (BF, 128, 36, 2), (BF, 256, 3, 3), (F32, 64, 4, 2)])
def test_scores_that_are_infinite(jb, new, kv, dtype, D, H, Hkv):
    """Infinite queries, keys and means: a score is what the products' sum is, an infinity of its sign
    or, of both signs or an infinity times 0, NaN.  (Sequence 1 has infinite queries, 2 an infinite key
    in its own page and means of pages before it.)"""
    page, G = 16, H // Hkv
    d, g = inputs(new, kv, H, Hkv, D, page, dtype, 16 if dtype == BF else 32, seed=D + H)
    first = np.concatenate([[0], np.cumsum(new)])
    inf = float("inf")
    d["q"][first[1], 0, 3] = inf                        # head 0 of key head 0
    d["q"][first[2] - 1, 0, 5], d["q"][first[2] - 1, H - 1, 6] = -inf, inf
    d["q"][first[2]:, H - G:, 9], d["q"][first[2]:, H - G:, 10] = 0.125, -0.5
    d["k_cache"][int(d["table"][2, (kv[2] - 1) // page]), 0, 0, 2] = inf
    means = f64(d["k_cache"]).mean(2)
    means[int(d["table"][1, 4]), 0, 3] = 0.0            # an infinite query times 0
    means[int(d["table"][1, 7]), 0, 3] = 0.5            # times a value of one part
    means[int(d["table"][2, 5]), Hkv - 1, 9] = -inf
    means[int(d["table"][2, 6]), Hkv - 1, 9:11] = inf, -inf
    means[int(d["table"][2, 7]), Hkv - 1, 9:11] = inf
    means[int(d["table"][2, 8]), Hkv - 1, 9] = 3.395e38  # rounds to an infinity in bf16
    m = torch.from_numpy(means).float().cuda()
    r = jb.block_scores(d["q"].cuda(), d["k_cache"].cuda(), m, g["table"], g["kv"], cu_seqlens=g["cu"])
    q, got_m = f64(d["q"]), f64(m)
    want = np.full((len(q), Hkv, d["table"].shape[1]), -inf)
    slack = np.zeros_like(want)
    with np.errstate(invalid="ignore"):
        for t, b, p in places(new, kv):
            for h in range(Hkv):
                for j in range(p // page + 1):
                    x = q[t, h * G:(h + 1) * G] * got_m[int(d["table"][b, j]), h]
                    want[t, h, j], slack[t, h, j] = x.sum(1).max(), (3 * D + 2) * 2.0 ** -24 * np.abs(x).sum(1).max()
    seen = [want[first[i]:first[i + 1]] for i in (1, 2)]
    assert all(np.isnan(x).any() and np.isposinf(x).any() for x in seen) and (G > 1 or np.isneginf(seen[0][0, 0, :100]).any())
    got = same_kind(r["scores"], want)
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= slack[fine]).all()



# --------------------------------------------------------------- selection


@pytest.mark.parametrize("width", [1, 63, 64, 65, 255, 256, 257, 1000, 1024, 1025, 4096, 5000, 16384, 20000])
@pytest.mark.parametrize("count,first,recent", [(1, 0, 1), (5, 2, 2), (64, 1, 1), (300, 0, 3)])
def test_select(jb, width, count, first, recent):
    """Random scores with many ties, infinities, NaN, zeros of both signs; tokens from the first
    row on, at every place of a page."""
    print(f"[select {width} {count} {first} {recent}]", flush=True)
    g = torch.Generator().manual_seed(width + count)
    page, Hkv, n = 16, 2, 7
    rows = sorted({0, 15, width * 16 - 1, width * 8, max(0, width * 16 - 17), min(width, count) * 16 - 1, min(width, count + 1) * 16 - 1})
    n = len(rows)
    x = torch.randn(n, Hkv, width, generator=g)
    x[:, 1] = (x[:, 1] * 2).round() / 2  # ties, +-0
    odd = torch.rand(n, Hkv, width, generator=g)
    x[odd < 0.05], x[odd > 0.95], x[(odd > 0.5) & (odd < 0.53)] = float("nan"), -float("inf"), float("inf")
    kv = torch.tensor([r + 1 for r in rows], dtype=torch.int32)
    got = jb.block_select(x.cuda(), kv.cuda(), count, page, first=first, recent=recent).cpu()
    for i, r in enumerate(rows):
        for h in range(Hkv):
            assert got[i, h].tolist() == ref8.select(x[i, h].tolist(), r // page, count, first, recent), (r, h)


def test_select_packed(jb):
    """Sequences of many lengths, tokens without rows, rows behind the last sequence and behind
    max_seqlen left as they are."""
    new, kv, page, Hkv, width = [4, 3, 0, 1, 70, 1], [2, 0, 9, 0, 400, 5], 16, 3, 30
    n = sum(new)
    x = torch.randn(n + 2, Hkv, width, generator=torch.Generator().manual_seed(0))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    for limit in (None, 40):
        out = torch.full((n + 2, Hkv, 6), 77, dtype=torch.int32, device="cuda")
        got = jb.block_select(x.cuda(), torch.tensor(kv, dtype=torch.int32).cuda(), 6, page, cu_seqlens=cu,
                              max_seqlen=limit, blocks=out).cpu()
        taken = set()
        for t, b, p in places(new, kv, limit):
            taken.add(t)
            for h in range(Hkv):
                want = ref8.select(x[t, h].tolist(), p // page, 6, 1, 1) if p >= 0 else [-1] * 6
                assert got[t, h].tolist() == want, (t, h)
        for t in set(range(n + 2)) - taken:
            assert (got[t] == 77).all()


# --------------------------------------------------------------- attention


def check_blocks(d, r, lists, new, kv, tokens=None, out=None):
    """r against the oracle over the rows of the pages that count."""
    H, D = d["q"].shape[-2:]
    Hkv, page = d["k_cache"].shape[1:3]
    q, o, lse = f64(d["q"]).reshape(-1, H, D), f64(r["o"]).reshape(-1, H, D), f64(r["lse"]).reshape(-1, H)
    assert not np.isnan(o[:sum(new)]).any() and not np.isnan(lse[:sum(new)]).any()
    kc, vc = f64(d["k_cache"]), f64(d["v_cache"])
    G, bf = H // Hkv, d["q"].dtype == BF
    lists = np.asarray(lists).reshape(-1, Hkv, np.asarray(lists).shape[-1])
    for t, b, p in places(new, kv, tokens):
        table = d["table"][b].tolist()
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            rows = [j * page + i for j in ref8.counting(lists[t, h].tolist(), p // page) for i in range(page) if j * page + i <= p]
            if not rows:
                assert (o[t, heads] == 0).all() and (lse[t, heads] == -np.inf).all(), (t, h)
                continue
            full = [ref.gather(c[:, h:h + 1], table, p + 1)[rows] for c in (kc, vc)]
            eo, el, mag, big = ref.attend(q[t:t + 1, heads], *full)
            ds = (D + 2) * 2.0 ** -24 * big
            tol = mag * ((2.0 ** -8 if bf and G > 32 else 2.0 ** -15 if bf else 0.0) + 2 * ds[..., None] + 2.0 ** -17)
            if r["o"].dtype == BF:
                tol = tol + 2.0 ** -8 * (np.abs(eo) + tol)
            assert (np.abs(o[t, heads] - eo[0]) <= tol[0]).all(), (t, h, np.abs(o[t, heads] - eo[0]).max())
            assert (np.abs(lse[t, heads] - el[0]) <= ds[0] + 2.0 ** -17 * (1 + np.abs(el[0]))).all(), (t, h)


def attend(jb, g, lists, **kw):
    r = jb.attn_blocks(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], lists.cuda(), k_scales=g["k_scales"],
                       v_scales=g["v_scales"], cu_seqlens=g["cu"], want_lse=True, **kw)
    torch.cuda.synchronize()
    return r


def some_lists(new, kv, Hkv, page, count, seed):
    g = np.random.default_rng(seed)
    out = np.full((sum(new), Hkv, count), -1, np.int32)
    for t, b, p in places(new, kv):
        for h in range(Hkv):
            if p >= 0:
                own = p // page
                n = int(g.integers(0, min(count, own + 1) + 1))
                out[t, h, :n] = np.sort(g.choice(own + 1, n, replace=False))
    return torch.from_numpy(out)


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("D,H,Hkv,page,count", [(128, 12, 2, 64, 3), (64, 5, 5, 16, 7), (256, 8, 2, 32, 2), (64, 40, 1, 16, 4)])
@pytest.mark.parametrize("dtype,bits", CACHES)
def test_attention(jb, lengths, dtype, bits, D, H, Hkv, page, count):
    new, kv = LENGTHS[lengths]
    print(f"[blocks {lengths} {dtype} {bits} D={D} H={H}/{Hkv} page={page} count={count}]", flush=True)
    d, g = inputs(new, kv, H, Hkv, D, page, dtype, bits, seed=D + H)
    lists = some_lists(new, kv, Hkv, page, count, seed=H)
    check_blocks(d, attend(jb, g, lists), lists, new, kv)


@pytest.mark.parametrize("dtype,bits", CACHES)
@pytest.mark.parametrize("B,count", [(3, 40), (2100, 2)])
def test_decode(jb, dtype, bits, B, count):
    """Long lists cut into runs, and thousands of units."""
    kv = [1 + (37 * b) % (1900 if B < 10 else 60) for b in range(B)]
    kv[0] = 1900 if B < 10 else 60
    d, g = inputs([1] * B, kv, 8, 2, 64, 16, dtype, bits, seed=B, packed=False)
    g["q"] = g["q"][:, 0]
    lists = some_lists([1] * B, kv, 2, 16, count, seed=B)
    lists[0, :, :] = torch.arange(min(count, 40))  # (more than kv[0] may have)
    check_blocks(d, attend(jb, g, lists, out_dtype=F32), lists, [1] * B, kv)


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_lists_that_do_not_ascend(jb, dtype, bits):
    """Entries out of range, twice, out of order, behind the token's page: passed over."""
    new, kv = [2, 1], [100, 33]
    d, g = inputs(new, kv, 4, 2, 64, 16, dtype, bits, seed=5)
    lists = torch.tensor([[[3, 3, 1, 5], [-1, 2, 2, 6]], [[0, 1000000, 6, 6], [6, 0, 1, 2]],
                          [[2, 0, 1, 2], [-5, -2147483648, 2147483647, 3]]], dtype=torch.int32)
    check_blocks(d, attend(jb, g, lists), lists, new, kv)


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_what_is_not_listed(jb, dtype, bits):
    """Rows that are not listed or lie behind the token change no bit, whatever they hold; a page
    out of range reads as zeros."""
    new, kv = [1, 3], [90, 61]
    d, g = inputs(new, kv, 4, 2, 64, 16, dtype, bits, seed=6)
    d["table"][0, 2] = 1 << 20
    g["table"] = d["table"].cuda()
    lists = torch.tensor([[[0, 2, 5, -1]] * 2, [[1, 3, -1, -1]] * 2, [[0, 3, -1, -1]] * 2, [[0, 1, 3, -1]] * 2], dtype=torch.int32)
    clean = attend(jb, g, lists)
    check_blocks(d, clean, lists, new, kv)
    seen = {(int(d["table"][b, j])) for t, b, p in places(new, kv) for j in lists[t, 0].tolist() if j >= 0}
    for x in ("k_cache", "v_cache"):
        for p in range(len(d[x])):
            if p not in seen:
                (g[x].view(torch.uint8) if bits == 8 else g[x])[p] = 0x7f if bits == 8 else float("nan")
        last = int(d["table"][0, 5])
        (g[x].view(torch.uint8) if bits == 8 else g[x])[last, :, 90 - 80:] = 0xff if bits == 8 else float("inf")
    dirty = attend(jb, g, lists)
    assert torch.equal(clean["o"], dirty["o"]) and torch.equal(clean["lse"], dirty["lse"])


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_rows_of_nobody_stay(jb, dtype, bits):
    """Rows behind the last sequence and behind max_seqlen."""
    new, kv = [50, 3], [70, 40]
    d, g = inputs(new, kv, 4, 2, 64, 16, dtype, bits, seed=7, behind=4)
    lists = torch.cat([some_lists(new, kv, 2, 16, 3, 1), torch.zeros(4, 2, 3, dtype=torch.int32)])
    for limit, stay in ((None, [*range(53, 57)]), (30, [*range(30, 50), *range(53, 57)])):
        o = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
        lse = torch.full(d["q"].shape[:-1], 5.0, device="cuda")
        r = attend(jb, g, lists, max_seqlen=limit, o=o, lse=lse)
        assert (r["o"][stay] == 5).all() and (r["lse"][stay] == 5).all()
        check_blocks(d, r, lists, new, kv, tokens=limit)


def test_q_strides_and_scale(jb):
    new, kv = [9], [200]
    d, g = inputs(new, kv, 6, 3, 128, 16, BF, 8, seed=8)
    wide = torch.randn(9, 8, 128, device="cuda").to(BF)
    wide[:, 1:7] = g["q"]
    lists = some_lists(new, kv, 3, 16, 5, 2)
    a = attend(jb, dict(g, q=wide[:, 1:7]), lists, scale=0.2)
    b = attend(jb, g, lists, scale=0.2)
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    means = torch.zeros(len(d["k_cache"]), 3, 128, device="cuda")
    args = (g["k_cache"], means, g["table"], g["kv"])
    x = [jb.block_scores(q, *args, k_scales=g["k_scales"], cu_seqlens=g["cu"])["scores"] for q in (wide[:, 1:7], g["q"])]
    assert torch.equal(x[0], x[1])


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_layer_at_a_long_context(jb, dtype, bits):
    """A prompt in chunks and decode steps of a packed batch: append, scores, selection and attention
    over the selected pages, each checked from what it was given; while a token sees no more pages
    than it may list, the result is that of the attention over the whole cache."""
    H, Hkv, D, page, count, B, pages = 4, 2, 64, 16, 4, 2, 12
    g = torch.Generator().manual_seed(bits)
    pool = B * pages + 1
    table = torch.randperm(pool, generator=g)[:B * pages].view(B, pages).to(torch.int32)
    kc, vc = (torch.zeros(pool, Hkv, page, D, dtype=torch.uint8 if bits == 8 else dtype).cuda() for _ in range(2))
    ks = vs = None
    if bits == 8:
        kc, vc = kc.view(E4M3), vc.view(E4M3)
        ks, vs = (torch.zeros(pool, Hkv, page // 16, dtype=torch.uint8).cuda().view(E8M0) for _ in range(2))
    means = torch.zeros(pool, Hkv, D).cuda()
    f = torch.tensor(1e4 ** (-np.arange(0, D, 2) / D), dtype=torch.float32).cuda()
    have = [0, 0]
    for new in ([37, 20], [40, 1], [1, 33], [1, 1], [1, 1], [50, 1]):
        kv = [h + t for h, t in zip(have, new)]
        n = sum(new)
        q, k, v = (torch.randn(n, h, D, generator=g).to(dtype) for h in (H, Hkv, Hkv))
        cu = torch.tensor([0, new[0], n], dtype=torch.int32).cuda()
        tab, lens = table.cuda(), torch.tensor(kv, dtype=torch.int32).cuda()
        if bits == 8:
            a = jb.qk_norm_rope_paged8(q.cuda(), k.cuda(), v.cuda(), kc, vc, ks, vs, tab, lens, f, cu_seqlens=cu)
        else:
            a = jb.qk_norm_rope_paged(q.cuda(), k.cuda(), v.cuda(), kc, vc, tab, lens, f, cu_seqlens=cu)
        s = jb.block_scores(a["q"], kc, means, tab, lens, k_scales=ks, cu_seqlens=cu)["scores"]
        lists = jb.block_select(s, lens, count, page, cu_seqlens=cu)
        r = jb.attn_blocks(a["q"], kc, vc, tab, lens, lists, k_scales=ks, v_scales=vs, cu_seqlens=cu, want_lse=True)
        whole = jb.attn_paged8(a["q"], kc, vc, ks, vs, tab, lens, cu_seqlens=cu, out_dtype=F32) if bits == 8 else \
            jb.attn_paged(a["q"], kc, vc, tab, lens, cu_seqlens=cu, out_dtype=F32)
        torch.cuda.synchronize()
        held = {"q": a["q"].cpu(), "table": table}
        for x, c, e in (("k_cache", kc, ks), ("v_cache", vc, vs)):
            held[x] = torch.from_numpy(ref8.dequantise(codes_of(c), codes_of(e))).float() if bits == 8 else c.cpu()
        x = s.cpu()
        keys = f64(held["k_cache"])
        for t, b, p in places(new, kv):
            own = p // page
            for h in range(Hkv):
                assert lists[t, h].tolist() == ref8.select(x[t, h].tolist(), own, count, 1, 1)
                m = np.stack([keys[int(table[b, j]), h, :min(page, kv[b] - j * page)].mean(0) for j in range(own + 1)])
                qs = f64(held["q"][t, h * 2:h * 2 + 2])
                slack = (3 * D + 2 + page + 1) * 2.0 ** -24 * np.abs(qs).sum(-1).max() * np.abs(m).max()
                slack += 2.0 ** -23 * np.abs(qs).sum(-1).max() * np.abs(keys).max() * page
                assert (np.abs(x[t, h, :own + 1].numpy() - (qs @ m.T).max(0)) <= slack).all()
            if own < count:
                off = (r["o"][t].float() - whole["o"][t]).abs().max().item()
                assert off <= 2.0 ** -7 * f64(held["v_cache"]).__abs__().max()
        check_blocks(held, r, lists.cpu(), new, kv)
        have = kv


def test_graph_of_a_step(jb):
    """Scores, selection and attention captured: every replay over new inputs, with eager calls
    between, gives the eager result; two graphs with workspaces of their own do not meet."""
    B, kv = 5, [900, 33, 1, 640, 200]
    d, g = inputs([1] * B, kv, 12, 2, 128, 16, BF, 8, seed=13, packed=False)
    q = g["q"][:, 0].contiguous()
    m0 = torch.from_numpy(f64(d["k_cache"]).mean(2)).float().cuda()

    def step(means):
        s = jb.block_scores(q, g["k_cache"], means, g["table"], g["kv"], k_scales=g["k_scales"])["scores"]
        lists = jb.block_select(s, g["kv"], 9, 16, first=1, recent=2)
        return lists, jb.attn_blocks(q, g["k_cache"], g["v_cache"], g["table"], g["kv"], lists, k_scales=g["k_scales"],
                                     v_scales=g["v_scales"], want_lse=True)

    means = [m0.clone() for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(means[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(means[i]))
    for k in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(k)).to(BF))
        for x in graphs:
            x.replay()
        want = step(means[2])
        torch.cuda.synchronize()
        for lists, r in outs:
            assert torch.equal(lists, want[0])
            assert torch.equal(r["o"], want[1]["o"]) and torch.equal(r["lse"], want[1]["lse"])


def test_another_stream(jb):
    """The calls run on the stream they are given."""
    kv = [500, 70]
    d, g = inputs([1, 1], kv, 8, 2, 64, 16, BF, 16, seed=14, packed=False)
    g["q"] = g["q"][:, 0].contiguous()
    means = torch.from_numpy(f64(d["k_cache"]).mean(2)).float().cuda()
    s = jb.block_scores(g["q"], g["k_cache"], means, g["table"], g["kv"])["scores"]
    lists = jb.block_select(s, g["kv"], 4, 16)
    want = jb.attn_blocks(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], lists)["o"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s2 = jb.block_scores(g["q"], g["k_cache"], means, g["table"], g["kv"], stream=side)["scores"]
    l2 = jb.block_select(s2, g["kv"], 4, 16, stream=side)
    o2 = jb.attn_blocks(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], l2, stream=side.cuda_stream)["o"]
    side.synchronize()
    assert torch.equal(s, s2) and torch.equal(lists, l2) and torch.equal(want, o2)


# --------------------------------------------------------- what breaks easily


@pytest.mark.parametrize("dtype,bits", CACHES)
@pytest.mark.parametrize("H,Hkv,page", [(8, 1, 16), (6, 3, 32)])
def test_not_finite_in_a_page_of_some(jb, dtype, bits, H, Hkv, page):
    """Tokens next to each other are computed together: a value that is not finite in a page that
    some of them list reaches those and no others, and a row behind a token's own none before it."""
    new, kv, D = [7], [150], 64
    d, g = inputs(new, kv, H, Hkv, D, page, dtype, bits, seed=20)
    own = [(kv[0] - 7 + i) // page for i in range(7)]
    lists = torch.tensor([[[0, 2 if t % 2 else 1, own[t], -1]] * Hkv for t in range(7)], dtype=torch.int32)
    clean = attend(jb, g, lists)
    check_blocks(d, clean, lists, new, kv)
    vc = g["v_cache"].view(torch.uint8) if bits == 8 else g["v_cache"]
    vc[int(d["table"][0, 2]), 0, 3, 40] = 0x7f if bits == 8 else float("inf")      # page 2: the odd tokens'
    last = 149
    vc[int(d["table"][0, last // page]), Hkv - 1, last % page, 9] = 0xff if bits == 8 else float("nan")  # the last token's row
    dirty = attend(jb, g, lists)
    G = H // Hkv
    want = torch.zeros(7, H, D, dtype=torch.bool)
    want[1::2, :G, 40] = True
    want[6, H - G:, 9] = True
    got = ~torch.isfinite(dirty["o"].float()).cpu()
    assert torch.equal(got, want)
    # (the second, careful pass takes the same steps)
    assert torch.equal(dirty["o"].cpu()[~want], clean["o"].cpu()[~want]) and torch.equal(dirty["lse"], clean["lse"])


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_lists_that_go_through_memory(jb, dtype, bits):
    """Lists longer than LDS holds, and tables too wide to merge tokens' lists."""
    for T, kv, count, width in ((1, 300, 2100, 40), (5, 300, 3, 5000), (5, 300, 2100, 5000)):
        d, g = inputs([T], [kv], 4, 2, 64, 16, dtype, bits, seed=count, packed=False)
        d["table"] = torch.cat([d["table"], torch.full((1, width - d["table"].shape[1]), -3, dtype=torch.int32)], 1)
        g["table"] = d["table"].cuda()
        lists = torch.full((T, 2, count), -1, dtype=torch.int32)
        lists[:, :, :3] = some_lists([T], [kv], 2, 16, 3, 4)
        lists[0, 0, :19] = torch.arange(19)[:count] if count >= 19 else lists[0, 0, :19]
        shaped = lists.view(1, T, 2, count)
        check_blocks(d, attend(jb, g, shaped), lists, [T], [kv])


@pytest.mark.parametrize("dtype,bits", CACHES)
@pytest.mark.parametrize("T", [2, 3, 17])
def test_dense_batches_of_several_tokens(jb, dtype, bits, T):
    kv = [40, T - 1, 333, 64]
    d, g = inputs([T] * 4, kv, 8, 2, 128, 32, dtype, bits, seed=T, packed=False)
    lists = some_lists([T] * 4, kv, 2, 32, 5, T)
    check_blocks(d, attend(jb, g, lists.view(4, T, 2, 5)), lists, [T] * 4, kv)


def test_packed_decode(jb):
    """One token a sequence, packed, with an empty sequence and rows behind the last one: scores,
    selection and attention are those of the dense batch."""
    new, kv = [1, 0, 1, 1], [100, 50, 17, 640]
    d, g = inputs(new, kv, 6, 2, 128, 16, BF, 8, seed=30, behind=1)
    keep = [0, 2, 3]
    means = [torch.from_numpy(f64(d["k_cache"]).mean(2)).float().cuda() for _ in range(2)]
    s = torch.full((4, 2, d["table"].shape[1]), 7.0, device="cuda")
    jb.block_scores(g["q"], g["k_cache"], means[0], g["table"], g["kv"], k_scales=g["k_scales"], cu_seqlens=g["cu"],
                    max_seqlen=1, scores=s)
    args = (g["table"][keep].contiguous(), g["kv"][keep].contiguous())
    want = jb.block_scores(g["q"][:3], g["k_cache"], means[1], *args, k_scales=g["k_scales"])["scores"]
    assert torch.equal(s[:3], want) and (s[3] == 7).all() and torch.equal(means[0], means[1])
    lists = torch.full((4, 2, 4), 9, dtype=torch.int32, device="cuda")
    jb.block_select(s, g["kv"], 4, 16, cu_seqlens=g["cu"], max_seqlen=1, blocks=lists)
    want = jb.block_select(want, args[1], 4, 16)
    assert torch.equal(lists[:3], want) and (lists[3] == 9).all()
    o = torch.full_like(g["q"], 3.0)
    jb.attn_blocks(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], lists, k_scales=g["k_scales"],
                   v_scales=g["v_scales"], cu_seqlens=g["cu"], max_seqlen=1, o=o)
    want = jb.attn_blocks(g["q"][:3], g["k_cache"], g["v_cache"], *args, want, k_scales=g["k_scales"],
                          v_scales=g["v_scales"])["o"]
    assert torch.equal(o[:3], want) and (o[3] == 3).all()


@pytest.mark.parametrize("H,Hkv,D", [(40, 2, 64), (17, 1, 256), (64, 1, 128)])
def test_scores_of_many_heads(jb, H, Hkv, D):
    """More query heads to a key head than a product has rows."""
    for T in (1, 5):
        d, g = inputs([T], [500], H, Hkv, D, 16, BF, 16, seed=H + T, packed=False)
        means = torch.from_numpy(f64(d["k_cache"]).mean(2)).float().cuda()
        got = f64(jb.block_scores(g["q"], g["k_cache"], means, g["table"], g["kv"])["scores"]).reshape(T, Hkv, -1)
        q, m, G = f64(d["q"]).reshape(T, H, D), f64(means), H // Hkv
        for i in range(T):
            own = (500 - T + i) // 16
            for h in range(Hkv):
                ms, qs = m[d["table"][0, :own + 1].numpy(), h], q[i, h * G:(h + 1) * G]
                slack = (3 * D + 2) * 2.0 ** -24 * (np.abs(qs) @ np.abs(ms).T).max(0)
                assert (np.abs(got[i, h, :own + 1] - (qs @ ms.T).max(0)) <= slack).all()
                assert (got[i, h, own + 1:] == -np.inf).all()


def test_select_at_the_widest(jb):
    """65536 pages, the most there may be; all scores equal; descending ones."""
    page, width, count = 16, 65536, 40
    kv = torch.tensor([page * width, page * 40000 + 3], dtype=torch.int32)
    for x in (torch.zeros(2, 1, width), -torch.arange(width, dtype=torch.float32).expand(2, 1, width).contiguous(),
              torch.randn(2, 1, width, generator=torch.Generator().manual_seed(1))):
        got = jb.block_select(x.cuda(), kv.cuda(), count, page, first=2, recent=3).cpu()
        for i in range(2):
            own = (int(kv[i]) - 1) // page
            assert got[i, 0].tolist() == ref8.select(x[i, 0].tolist(), own, count, 2, 3)
