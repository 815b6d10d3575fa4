"""GPU parity of jb_attn_paged with the fp64 oracle (oracle/attention.py): chunks, packed
batches, decode, windows, empty rows, page sizes, strides, non-finite values where no query
looks, malformed device-side indices, streams and captured graphs.

Bounds, per element: the softmax weights are rounded to bf16 (half a step, 2^-8 of each), so
o is off by at most 2^-8 sum w |v|; a bf16 o by another 2^-8 |o|.  A score is off by at most
(D + 2) 2^-24 sum |q_d k_d| scale (fp32 sums of exact products, one scaling), which moves every
weight by that relative amount, up and down (numerator and denominator: twice); exp2, its
argument and the sums add less than 2^-17."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def jb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def batch(new, kv, H, Hkv, D, page, dtype, seed=0, packed=True, extra_pages=2, behind=0):
    """Inputs on the CPU: q packed (with `behind` rows after the last sequence) or [B, T, H, D],
    caches with every sequence's pages anywhere."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-l // page) for l in kv]
    pool = sum(need) + extra_pages
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.zeros(len(kv), max(max(need), 1), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    n = sum(new)
    q = torch.randn(n + behind, H, D, generator=g).to(dtype)
    d = dict(q=q if packed else q.view(len(new), new[0], H, D),
             k_cache=torch.randn(pool, Hkv, page, D, generator=g).to(dtype),
             v_cache=torch.randn(pool, Hkv, page, D, generator=g).to(dtype), table=table,
             kv=torch.tensor(kv, dtype=torch.int32), cu=None)
    if packed:
        d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return d


def call(jb, d, **kw):
    g = {k: None if v is None else v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    r = jb.attn_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], cu_seqlens=g["cu"], want_lse=True, **kw)
    torch.cuda.synchronize()
    return r


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(d, r, new, kv, window=0, scale=None, tokens=None):
    """r against the oracle, sequence by sequence (tokens: {sequence: tokens to look at})."""
    H, D = d["q"].shape[-2:]
    bf = d["q"].dtype == BF
    q, o, lse = f64(d["q"]).reshape(-1, H, D), f64(r["o"]).reshape(-1, H, D), f64(r["lse"]).reshape(-1, H)
    kc, vc = f64(d["k_cache"]), f64(d["v_cache"])
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        k, v = ref.gather(kc, d["table"][b].tolist(), l), ref.gather(vc, d["table"][b].tolist(), l)
        first = 0 if tokens is None else max(0, t - tokens)
        eo, el, mag, big = ref.attend(q[at + first:at + t], k, v, window, scale)
        go, gl = o[at + first:at + t], lse[at + first:at + t]
        ds = (D + 2) * 2.0 ** -24 * big
        tol = mag * ((2.0 ** -8 if bf else 0.0) + 2 * ds[..., None] + 2.0 ** -17)
        if r["o"].dtype == BF:
            tol = tol + 2.0 ** -8 * (np.abs(eo) + tol)
        bad = np.abs(go - eo) > tol
        assert not bad.any(), (b, t, l, np.argwhere(bad)[:3].tolist(), np.abs(go - eo).max())
        seen = np.isfinite(el)
        assert np.array_equal(gl == -np.inf, ~seen), b
        assert (np.abs(gl[seen] - el[seen]) <= ds[seen] + 2.0 ** -17 * (1 + np.abs(el[seen]))).all(), b
        at += t


# new tokens and cache rows of each sequence
LENGTHS = {
    "edges": ([1, 2, 5, 31, 33, 64, 65, 130], [1, 64, 65, 31, 127, 128, 65, 300]),
    "empty rows": ([4, 3, 0, 1, 70, 1], [2, 0, 9, 0, 40, 5]),   # more new tokens than rows; no rows; no tokens
    "mix": ([1, 1, 200, 1, 90], [700, 33, 513, 64, 90]),
}


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,D,H,Hkv,page,window", [
    (BF, 128, 12, 2, 64, 0), (BF, 128, 4, 4, 16, 100), (BF, 64, 8, 1, 32, 0), (BF, 64, 5, 5, 128, 33),
    (BF, 256, 4, 2, 16, 0), (BF, 256, 8, 1, 64, 70), (F32, 64, 6, 3, 16, 0), (F32, 128, 4, 1, 32, 50),
    (F32, 256, 2, 1, 16, 0),
])
def test_packed(jb, lengths, dtype, D, H, Hkv, page, window):
    new, kv = LENGTHS[lengths]
    print(f"[attn {lengths} {dtype} D={D} H={H}/{Hkv} page={page} window={window}]", flush=True)
    d = batch(new, kv, H, Hkv, D, page, dtype, seed=D + H)
    check(d, call(jb, d, window=window), new, kv, window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_seqlen,max_kv", [(None, None), (200, 16), (200, 1 << 20)])
def test_plan_hints_change_no_result(jb, dtype, max_seqlen, max_kv):
    """One piece of the cache, or many: the same rows, whatever the planned lengths."""
    new, kv = [200, 1, 64], [2000, 1500, 64]
    d = batch(new, kv, 6, 2, 64, 16, dtype, seed=3)
    # a table with room for more pages than the sequences have
    d["table"] = torch.cat([d["table"], torch.full((3, 200), -1, dtype=torch.int32)], 1)
    check(d, call(jb, d, max_seqlen=max_seqlen, max_kv=max_kv), new, kv)


@pytest.mark.parametrize("D,H,Hkv,T", [(128, 12, 2, 1), (128, 16, 2, 3), (64, 32, 1, 1), (64, 40, 1, 1), (256, 8, 2, 1)])
@pytest.mark.parametrize("out", [BF, F32])
def test_decode(jb, D, H, Hkv, T, out):
    """Single tokens (and three) of each sequence, dense; 40 query heads to a key head pass the
    32 rows of the decode kernel."""
    kv = [T, 17, 4096, 1000, 2049]
    new = [T] * 5
    d = batch(new, kv, H, Hkv, D, 32, BF, seed=T, packed=False)
    if T == 1:
        d["q"] = d["q"][:, 0]
    check(d, call(jb, d, out_dtype=out), new, kv)


@pytest.mark.parametrize("window", [0, 1152])
def test_chunk_at_the_end_of_a_long_context(jb, window):
    new, kv = [300], [20000]
    d = batch(new, kv, 12, 2, 128, 64, BF, seed=8)
    check(d, call(jb, d, window=window), new, kv, window, tokens=3)


def test_scale_and_large_scores(jb):
    """A scale of its own, and scores of both signs up to some hundreds: the running maximum
    moves, and weights underflow to zero."""
    new, kv = [40, 1], [400, 333]
    d = batch(new, kv, 4, 2, 128, 16, BF, seed=4)
    check(d, call(jb, d, scale=0.5), new, kv, scale=0.5)
    d["q"] = d["q"] * 30
    check(d, call(jb, d), new, kv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_that_no_query_sees(jb, dtype, bad):
    """Rows behind the cache's end in its last page, rows before every window, pages no table
    names; and new tokens' own rows, which earlier tokens must not feel."""
    new, kv, page, window = [50, 1, 3], [150, 101, 230], 32, 64
    d = batch(new, kv, 6, 2, 64, page, dtype, seed=5)
    clean = call(jb, d, window=window)
    for b, l in enumerate(kv):
        first = l - new[b]
        for c in ("k_cache", "v_cache"):
            last = int(d["table"][b, (l - 1) // page])
            d[c][last, :, (l - 1) % page + 1:] = bad          # behind the end
            for j in range(max(0, first - window + 1)):       # before the first query's window
                d[c][int(d["table"][b, j // page]), :, j % page] = bad
    used = set(int(p) for b, l in enumerate(kv) for p in d["table"][b, :-(-l // page)])
    for p in set(range(d["k_cache"].shape[0])) - used:
        d["k_cache"][p] = d["v_cache"][p] = bad
    r = call(jb, d, window=window)
    assert torch.equal(r["o"], clean["o"]) and torch.equal(r["lse"], clean["lse"])
    # the value row of new token 20 of sequence 0: the 20 before it must not change beyond the
    # order of their sums
    j = kv[0] - new[0] + 20
    d["v_cache"][int(d["table"][0, j // page]), :, j % page] = bad
    r = call(jb, d, window=window)
    assert not torch.isfinite(r["o"][20:50].float()).any()
    sub = {k: v for k, v in r.items()}
    sub["o"], sub["lse"] = r["o"][:20], r["lse"][:20]
    dd = dict(d, q=d["q"][:20])
    # as a batch of its own: the first 20 tokens over the rows that end with them
    for c in ("k_cache", "v_cache"):
        dd[c] = torch.nan_to_num(d[c], nan=0.0, posinf=0.0, neginf=0.0)
    check(dd, sub, [20], [kv[0] - 30], window)
    # ... and of the last token of the one after: a decode row sees it
    assert torch.equal(r["o"][50:], clean["o"][50:])


def test_pages_out_of_range_read_as_zeros(jb):
    new, kv, page = [20, 1], [100, 90], 16
    for dtype in (BF, F32):
        d = batch(new, kv, 4, 2, 64, page, dtype, seed=6)
        d["table"][0, 1], d["table"][0, 6], d["table"][1, 3] = -1, 10 ** 9, d["k_cache"].shape[0]
        check(d, call(jb, d), new, kv)


def test_malformed_offsets_and_lengths_stay_in_bounds(jb):
    """cu_seqlens and kv_lens come from device memory: offsets past the rows, negative and
    decreasing ones, lengths past the table give wrong rows, but nothing outside o and lse is
    written (their guards keep their fill)."""
    print("[malformed cu_seqlens, kv_lens]", flush=True)
    H, D, n = 4, 64, 120
    for dtype in (BF, F32):
        d = batch([40, 40, 40], [60, 60, 60], H, 2, D, 16, dtype, seed=7)
        d["cu"] = torch.tensor([0, 500, -40, 120], dtype=torch.int32)
        d["kv"] = torch.tensor([10 ** 9, -5, 64], dtype=torch.int32)
        o = torch.full((n + 200, H, D), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((n + 200, H), 7.0, device="cuda")
        call(jb, d, o=o[100:100 + n], lse=lse[100:100 + n])
        for t in (o, lse):
            assert (t[:100] == 7).all() and (t[100 + n:] == 7).all()


@pytest.mark.parametrize("max_kv", [64, 1 << 16])
def test_rows_behind_the_last_sequence_stay(jb, max_kv):
    new, kv = [30, 1, 17], [300, 200, 17]
    for dtype in (BF, F32):
        d = batch(new, kv, 4, 2, 64, 16, dtype, seed=9, behind=21)
        o = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
        lse = torch.full(d["q"].shape[:2], 5.0, device="cuda")
        r = call(jb, d, o=o, lse=lse, max_kv=max_kv)
        check(dict(d, q=d["q"][:48]), dict(o=r["o"][:48], lse=r["lse"][:48]), new, kv)
        assert (o[48:] == 5).all() and (lse[48:] == 5).all()


def test_sequences_longer_than_planned_are_cut(jb):
    new, kv = [30, 90, 40], [300, 90, 200]
    d = batch(new, kv, 4, 2, 64, 16, BF, seed=10)
    o = torch.full(d["q"].shape, 5.0, dtype=BF, device="cuda")
    r = call(jb, d, o=o, max_seqlen=60)
    assert (o[30 + 60:30 + 90] == 5).all() and torch.isfinite(r["o"].float()).all()
    # the sequences that fit are as ever
    e = call(jb, d)
    assert torch.equal(r["o"][:30], e["o"][:30]) and torch.equal(r["o"][120:], e["o"][120:])


def test_strides(jb):
    """q as a slice of one projection's output, the caches as one layer of several."""
    new, kv, H, Hkv, D, page = [3, 50], [70, 50], 6, 2, 128, 16
    d = batch(new, kv, H, Hkv, D, page, BF, seed=11)
    e = call(jb, d)
    wide = torch.randn(53, H + 2 * Hkv, D).to(BF).cuda()
    wide[:, :H] = d["q"].cuda()
    P = d["k_cache"].shape[0]
    layers = torch.randn(P, 2, 3, Hkv, page, D).to(BF).cuda()   # [page][k, v][layer]
    layers[:, 0, 1], layers[:, 1, 1] = d["k_cache"].cuda(), d["v_cache"].cuda()
    r = jb.attn_paged(wide[:, :H], layers[:, 0, 1], layers[:, 1, 1], d["table"].cuda(), d["kv"].cuda(),
                      cu_seqlens=d["cu"].cuda(), want_lse=True)
    assert torch.equal(r["o"], e["o"]) and torch.equal(r["lse"], e["lse"])


def test_cache_past_32_bit_offsets(jb):
    """Pages whose offsets pass 2^32 bytes and 2^32 elements."""
    H, Hkv, D, page = 4, 2, 128, 64
    P = (1 << 32) // (Hkv * page * D) + 40
    new, kv = [1, 40], [200, 150]
    d = batch(new, kv, H, Hkv, D, page, BF, seed=12)
    big = [torch.empty(P, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2)]
    table = d["table"] + (P - d["k_cache"].shape[0])
    table[1] = d["table"][1] + (1 << 31) // (Hkv * page * D)
    for b, l in enumerate(kv):
        for x in range(-(-l // page)):
            big[0][int(table[b, x])] = d["k_cache"][int(d["table"][b, x])].cuda()
            big[1][int(table[b, x])] = d["v_cache"][int(d["table"][b, x])].cuda()
    r = jb.attn_paged(d["q"].cuda(), *big, table.cuda(), d["kv"].cuda(), cu_seqlens=d["cu"].cuda(), want_lse=True)
    check(d, r, new, kv)


def test_same_results_every_time_and_on_another_stream(jb):
    new, kv = [60, 1, 1], [5000, 4000, 77]
    d = batch(new, kv, 12, 2, 128, 64, BF, seed=13)
    e = call(jb, d)
    g = {k: v.cuda() for k, v in d.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            r = jb.attn_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], cu_seqlens=g["cu"], want_lse=True)
        s.synchronize()
        assert torch.equal(r["o"], e["o"]) and torch.equal(r["lse"], e["lse"])


def test_captured_graphs(jb):
    """A decode step and a chunk in graphs of their own, replayed with new contents and eager
    calls between."""
    for new, kv in (([1] * 3, [900, 64, 333]), ([70, 2], [900, 40])):
        d = batch(new, kv, 12, 2, 128, 64, BF, seed=14)
        g = {k: v.cuda() for k, v in d.items()}

        def go():
            return jb.attn_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], cu_seqlens=g["cu"],
                                 want_lse=True)
        go()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = go()
        for i in range(4):
            g["q"].copy_(torch.randn_like(g["q"].float()).to(BF))
            g["v_cache"].mul_(0.5)
            e = go()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out["o"], e["o"]) and torch.equal(out["lse"], e["lse"]), i


@pytest.mark.parametrize("B,packed", [(2100, False), (600, True), (300, True)])
def test_many_sequences(jb, B, packed):
    """Thousands of decode units (one each a workgroup), and hundreds in equal runs: sequences of
    no, one to three tokens and 0 to 700 rows in any order."""
    rng = np.random.RandomState(B)
    new = rng.randint(0, 4, B).tolist() if packed else [1] * B
    kv = rng.randint(0, 60 if B > 1000 else 700, B).tolist()
    d = batch(new, kv, 4, 2, 64, 16, BF, seed=B, packed=packed)
    check(d, call(jb, d, max_seqlen=3), new, kv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 3])
def test_256_queries_to_a_key_head(jb, dtype, T):
    """A token's rows fill two tiles of queries."""
    new, kv = [T, T], [200, 33]
    d = batch(new, kv, 256, 1, 64, 32, dtype, seed=15)
    check(d, call(jb, d), new, kv)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new", [[40, 1, 2], [2, 1, 3]])
def test_non_finite_value_between_new_tokens(jb, D, new):
    """A value row that only the later new tokens see (chunk and decode kernels, larger heads):
    theirs are not finite, the others' bits stay."""
    kv, page = [90, 70, 100], 16
    d = batch(new, kv, 4, 2, D, page, BF, seed=D)
    clean = call(jb, d)
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        if t > 1:
            j = l - 1   # the last new token's own row
            d["v_cache"][int(d["table"][b, j // page]), :, j % page, 5] = float("inf")
    r = call(jb, d)
    for b, t in enumerate(new):
        rows = slice(at, at + t - 1 if t > 1 else at + t)
        assert torch.equal(r["o"][rows], clean["o"][rows]) and torch.equal(r["lse"][rows], clean["lse"][rows]), b
        if t > 1:
            last = r["o"][at + t - 1].float()
            assert torch.isinf(last[:, 5]).all()
            keep = torch.arange(D, device="cuda") != 5
            assert torch.equal(last[:, keep], clean["o"][at + t - 1].float()[:, keep])
        at += t


@pytest.mark.parametrize("as_handle", [False, True])
def test_stream_argument(jb, as_handle):
    """The stream argument, a torch stream or its handle: the call and its allocations belong to
    it (the current stream may reuse nothing of them meanwhile)."""
    new, kv = [1] * 4, [9000, 5000, 77, 1000]
    d = batch(new, kv, 12, 2, 128, 64, BF, seed=16)
    e = call(jb, d)
    g = {k: v.cuda() for k, v in d.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        r = jb.attn_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], cu_seqlens=g["cu"],
                          stream=s.cuda_stream if as_handle else s)
        torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda")  # the current stream's own allocations
        s.synchronize()
        assert torch.equal(r["o"], e["o"])


def test_two_calls_at_once(jb):
    """Calls on two streams, each with a workspace of its own, do not touch each other."""
    s = [torch.cuda.Stream() for _ in range(2)]
    ds, es, gs = [], [], []
    for i, (new, kv) in enumerate((([1] * 3, [9000, 4000, 100]), ([300, 1], [3000, 2500]))):
        d = batch(new, kv, 12, 2, 128, 64, BF, seed=17 + i)
        es.append(call(jb, d))
        gs.append({k: v.cuda() for k, v in d.items()})
    torch.cuda.synchronize()
    for _ in range(4):
        rs = [jb.attn_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["kv"], cu_seqlens=g["cu"], stream=t)
              for g, t in zip(gs, s)]
        for t in s:
            t.synchronize()
        for r, e in zip(rs, es):
            assert torch.equal(r["o"], e["o"])


def test_first_offset_is_not_zero(jb):
    """Rows before the first sequence belong to nobody either."""
    new, kv = [30, 1], [100, 64]
    for dtype in (BF, F32):
        d = batch(new, kv, 4, 2, 64, 16, dtype, seed=19, behind=9)
        e = call(jb, d)
        d["q"] = torch.cat([d["q"][31:], d["q"][:31]])
        d["cu"] = d["cu"] + 9
        o = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
        r = call(jb, d, o=o)
        assert torch.equal(r["o"][9:], e["o"][:31]) and (o[:9] == 5).all()


def test_a_call_waits_for_its_stream(jb):
    """Inputs that the given stream writes late, behind long work: every call with that stream reads
    them as written (on the current stream it would find them too early)."""
    d = batch([1] * 3, [900, 400, 100], 12, 2, 128, 64, BF, seed=23)
    g = {k: v.cuda() for k, v in d.items()}
    x, k, v = g["q"], torch.randn(3, 2, 128, device="cuda").to(BF), torch.randn(3, 2, 128, device="cuda").to(BF)
    pos, fr = torch.arange(3, dtype=torch.int32, device="cuda"), torch.rand(64, device="cuda")
    tail = (g["k_cache"], g["v_cache"], g["table"], g["kv"])
    runs = [lambda q, **a: jb.qk_norm_rope(q, k, pos, fr, **a)[0],
            lambda q, **a: jb.qk_norm_rope_backward(q, k, pos, fr, torch.ones_like(q), k, **a)["dq"],
            lambda q, **a: jb.qk_norm_rope_paged(q, k, v, g["k_cache"].clone(), g["v_cache"].clone(), *tail[2:], fr, **a)["q"],
            lambda q, **a: jb.attn_paged(q, *tail, **a)["o"]]
    s, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device="cuda").to(BF)
    for i, run in enumerate(runs):
        print(f"[late input, call {i}]", flush=True)
        want, q = run(x), torch.zeros_like(x)
        run(q, stream=s)  # (allocations of the first call are behind us)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):
                busy @ busy
            q.copy_(x)
        got = run(q, stream=s)
        s.synchronize()
        assert torch.equal(got, want), i


@pytest.mark.parametrize("D,H,Hkv", [(256, 8, 8), (128, 32, 16), (64, 24, 24)])
@pytest.mark.parametrize("behind", [0, 77])
def test_last_round_in_pieces(jb, D, H, Hkv, behind):
    """A few more tiles than the chip takes at once, under a window: the ranges of the last ones
    are in pieces, the others whole.  Tokens from all over each sequence, and rows of nobody."""
    G = H // Hkv
    new, kv, window = [1500 // G, 0, 1300 // G, 1424 // G], [2600, 40, 1300, 1900], 1000
    d = batch(new, kv, H, Hkv, D, 64, BF, seed=D + behind, behind=behind)
    o = torch.full(d["q"].shape, 5.0, dtype=BF, device="cuda")
    shape = jb.AttnShape(4, max(new), H, Hkv, D, 0, 64, 41, d["k_cache"].shape[0], 2600, window,
                         jb.JB_BF16, jb.JB_BF16, 0, 0, 0, 0, 0)
    pieces = jb.attn_paged_workspace_size(shape, sum(new) + behind, True)
    assert 0 < pieces < 2 * (sum(new) + behind) * H * D * 4  # (all rows in pieces: that at least)
    r = call(jb, d, window=window, max_seqlen=max(new), max_kv=2600, o=o)
    assert (o[sum(new):] == 5).all()
    at = 0
    for b, t in enumerate(new):
        for i in sorted({0, 1, 63 // G, 126 // G, 200, t // 2, t - 131, t - 3}) if t else ():
            one = dict(d, q=d["q"][at + i:at + i + 3], table=d["table"][b:b + 1])
            check(one, dict(o=r["o"][at + i:at + i + 3], lse=r["lse"][at + i:at + i + 3]), [3], [kv[b] - t + i + 3], window)
        at += t
