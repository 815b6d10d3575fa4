"""GPU parity of the 8-bit cache's operators (jb_qk_norm_rope_paged8, jb_attn_paged8) with the fp64
oracles (oracle/attention.py, oracle/blocks.py): every append and attention over lengths, head
layouts, types and pages, blocks of 16 rows that several calls fill, codes and scales that are
not numbers, malformed device-side indices, strides, streams and captured graphs.

Bounds.  Values are copied exactly before they are rounded, so V's codes and scales are the
oracle's bit for bit.  A query's norm and turn, in fp32, are off by at most TURN of the row's
largest magnitude (a sum of D squares, a square root, a division, two products and a sum: less than
2^-20 with the sine's 1.5e-7).  A key's are in 64 bits where it counts; it is held to half a step of
its code and twice TURN here, and to its value in 64 bits at the codes' borders below (and in
test_gpu_long_edges).
The attention's bounds are test_gpu_attn's, on the values that the cache holds."""
import numpy as np
import pytest
import torch

from layer_checks import numbers
from oracle import attention as ref
from oracle import blocks as ref8
from test_gpu_attn import BF, F32, LENGTHS, batch, check, f64

pytestmark = pytest.mark.gpu
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TURN = 2.0 ** -20


@pytest.fixture(scope="module")
def jb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def codes_of(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def in_8_bits(cache, seed=0):
    """A cache's values in 8 bits: (codes, scales) uint8 arrays, scales of different sizes."""
    g = np.random.default_rng(seed)
    x = f64(cache)
    P, Hkv, page, D = x.shape
    blocks = x.reshape(P, Hkv, page // 16, 16, D)
    most = np.abs(blocks).max((-2, -1))
    e = np.vectorize(ref8.exponent)(most) + g.integers(0, 3, most.shape)
    codes = ref8.encode(blocks / ref8.scale_value(e)[..., None, None]).reshape(x.shape)
    return codes, e.astype(np.uint8)


def batch8(*args, **kw):
    """test_gpu_attn's batch with its caches in 8 bits, and with the values they hold."""
    d = batch(*args, **kw)
    d8 = dict(d)
    for x in ("k", "v"):
        codes, e = in_8_bits(d[x + "_cache"], seed=ord(x))
        d8[x + "_cache"], d8[x + "_scales"] = torch.from_numpy(codes).view(E4M3), torch.from_numpy(e).view(E8M0)
        d[x + "_cache"] = torch.from_numpy(ref8.dequantise(codes, e)).float()  # (exact)
    return d, d8


def on_gpu(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def call(jb, d8, **kw):
    g = on_gpu(d8)
    r = jb.attn_paged8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"],
                       cu_seqlens=g["cu"], want_lse=True, **kw)
    torch.cuda.synchronize()
    return r


def strict(d, r, new, kv, *args, **kw):
    numbers(r["o"], sum(new))
    numbers(r["lse"].unsqueeze(-1), sum(new))
    check(d, r, new, kv, *args, **kw)


# ------------------------------------------------------------------ append


def append_inputs(new, kv, H, Hkv, D, page, dtype, seed=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    d = batch8(new, kv, H, Hkv, D, page, dtype, seed=seed, behind=behind)[1]
    n = d["q"].shape[0]
    # rows of different sizes, some zero
    size = 2.0 ** torch.randint(-6, 7, (n, Hkv, 1), generator=g) * (torch.rand(n, Hkv, 1, generator=g) > 0.1)
    d["k"] = torch.randn(n, Hkv, D, generator=g).to(dtype)
    d["v"] = (torch.randn(n, Hkv, D, generator=g) * size).to(dtype)
    d["wq"] = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype)
    d["wk"] = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype)
    return d


def append(jb, d, inv_freq, **kw):
    g = on_gpu(d)
    r = jb.qk_norm_rope_paged8(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"],
                               g["kv"], inv_freq.cuda(), g["wq"], g["wk"], cu_seqlens=g["cu"], **kw)
    torch.cuda.synchronize()
    return r


def equal(got, want, nan=255):
    """The same codes (a NaN of either sign is the same)."""
    same = (np.where(got == nan, 127, got) == np.where(want == nan, 127, want))
    assert same.all(), (np.argwhere(~same)[:4].tolist(), got[~same][:4], want[~same][:4])


def check_append(d, r, new, kv, inv_freq, interleaved=False, tokens=None, offsets=None):
    """The queries, codes and scales after one append of d's rows to d's caches."""
    H, D = d["q"].shape[-2:]
    Hkv = d["k"].shape[-2]
    q, k, v = f64(d["q"]).reshape(-1, H, D), f64(d["k"]).reshape(-1, Hkv, D), f64(d["v"]).reshape(-1, Hkv, D)
    got_q = f64(r["q"]).reshape(-1, H, D)
    want = {x: (codes_of(d[x + "_cache"]).copy(), codes_of(d[x + "_scales"]).copy()) for x in ("k", "v")}
    keys = {}
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        m = t if tokens is None else min(t, tokens)
        rows = np.arange(l - t, l)
        eq = ref.norm_rope(q[at:at + t], rows, inv_freq.numpy(), f64(d["wq"]), interleaved=interleaved)
        ek = ref.norm_rope(k[at:at + t], rows, inv_freq.numpy(), f64(d["wk"]), interleaved=interleaved)
        tol = TURN * np.abs(eq).max(-1, keepdims=True) + (2.0 ** -8 if d["q"].dtype == BF else 0) * np.abs(eq)
        assert (np.abs(got_q[at:at + m] - eq[:m]) <= tol[:m]).all(), b
        table = d["table"][b].tolist()
        ref8.append(*want["v"], table, l, v[at:at + t], tokens)
        near = ref8.append(*want["k"], table, l, ek, tokens).values()
        assert all(n < 1 - 2 * TURN and (n > 0.5 + 2 * TURN or n == 0) for n in near), "a scale next to its border"
        page = d["k_cache"].shape[2]
        for i, row in enumerate(rows[:m]):
            if row >= 0 and 0 <= table[row // page] < len(want["k"][0]):
                keys[table[row // page], row % page] = ek[i]
        at += t
    equal(codes_of(r["v_cache"]), want["v"][0])
    equal(codes_of(r["v_scales"]), want["v"][1], nan=256)
    equal(codes_of(r["k_scales"]), want["k"][1], nan=256)
    got = codes_of(r["k_cache"])
    same = got == want["k"][0]
    for (p, row), y in keys.items():
        s = ref8.scale_value(want["k"][1][p, :, row // 16])[:, None]
        off = np.abs(ref8.E4M3[got[p, :, row]] * s - y)
        tol = TURN * np.abs(y).max(-1, keepdims=True)
        assert (off <= ref8.half_step(y / s) * s + 2 * tol).all(), (p, row)
        same[p, :, row] = True
    assert same.all(), np.argwhere(~same)[:4].tolist()


def frequencies(rot):
    return torch.tensor(1e4 ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32)


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,D,H,Hkv,page,rot,pairs", [
    (BF, 128, 12, 2, 64, 128, False), (BF, 64, 8, 1, 32, 32, True), (BF, 256, 4, 2, 16, 256, False),
    (F32, 64, 6, 3, 16, 64, False), (F32, 128, 4, 1, 128, 64, True), (F32, 256, 2, 1, 32, 256, True),
])
def test_append(jb, lengths, dtype, D, H, Hkv, page, rot, pairs):
    new, kv = LENGTHS[lengths]
    print(f"[append8 {lengths} {dtype} D={D} H={H}/{Hkv} page={page}]", flush=True)
    d = append_inputs(new, kv, H, Hkv, D, page, dtype, seed=D + H)
    f = frequencies(rot)
    check_append(d, append(jb, d, f, interleaved=pairs), new, kv, f, pairs)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 256)])
def test_append_row_by_row(jb, dtype, D):
    """Forty rows in steps of one to three: every block of 16 is filled by several calls, its scale
    grows and earlier codes shrink with it; each step is checked from the cache it found."""
    f = frequencies(D)
    d = append_inputs([3] * 2, [3, 3], 2, 2, D, 16, dtype, seed=1)
    d["table"] = torch.tensor([[3, 0, 1, -1], [2, 99, 4, 5]], dtype=torch.int32)  # some rows have no page
    d["k_cache"], d["v_cache"] = (torch.zeros(6, 2, 16, D, dtype=torch.uint8).view(E4M3) for _ in range(2))
    d["k_scales"], d["v_scales"] = (torch.full((6, 2, 1), 200, dtype=torch.uint8).view(E8M0) for _ in range(2))
    row, step = 0, 0
    while row < 40:
        t = 1 + step % 3
        x = append_inputs([t] * 2, [row + t] * 2, 2, 2, D, 16, dtype, seed=step)
        d.update({n: x[n] for n in ("q", "k", "v", "cu", "kv")})
        d["k"], d["v"] = d["k"] * (1 + step), d["v"] * (1 + step) ** 2  # (k's size goes in the norm)
        r = append(jb, d, f)
        check_append(d, r, [t] * 2, [row + t] * 2, f)
        for n in ("k_cache", "v_cache", "k_scales", "v_scales"):
            d[n] = r[n].cpu()
        row, step = row + t, step + 1


def test_append_not_finite(jb):
    """Infinities and NaN become NaN codes and have no part in the scale; a block of zeros has the
    smallest scale; the largest and smallest magnitudes of fp32 fit."""
    d = append_inputs([40], [45], 2, 1, 64, 16, F32, seed=2)
    v = d["v"]
    v[0], v[1, 0, 3], v[2, 0, 5], v[3, 0, 7] = 0, float("inf"), float("nan"), -float("inf")
    v[11:27] = 0  # rows 16 .. 31: a whole block
    v[27:] = torch.linspace(-3.4e38, 3.4e38, 13 * 64).view(13, 1, 64)
    f = frequencies(64)
    check_append(d, append(jb, d, f), [40], [45], f)
    d["v"][:] = 1e-41
    d["kv"][:] = 48  # from row 8 on: rows before them stay and hold the larger scale
    check_append(d, append(jb, d, f), [40], [48], f)


@pytest.mark.parametrize("dtype,D,pairs", [(BF, 128, False), (BF, 64, True), (F32, 128, True), (F32, 256, False)])
def test_append_codes_at_their_borders(jb, dtype, D, pairs):
    """A key's code is that of its value in 64 bits, but where the value lies nearer to a border than
    what the append is off by.  Of a cos + b sin the fp32 terms are at most 0.293 a, of y (3 half steps of
    2^-24) times a sum (2.3) and rounded, and 0.078 b, of f y (5) times a sum (2.5) and rounded twice;
    their sum, at most 0.37, is rounded once: 0.293 * 6.3 and 0.078 * 9.5 add up to 2 as a root of squares,
    with 0.37 and what the series leave out (0.04) 2.5 half steps of hypot(a, b).  The rest is in 64
    bits, and rounding to fp32 in between keeps the side of a border."""
    print(f"[append8 borders {dtype} D={D} pairs={pairs}]", flush=True)
    new, kv, Hkv, page = [1000, 1500], [1003, 1700], 2, 64
    d = append_inputs(new, kv, 2, Hkv, D, page, dtype, seed=D)
    f = frequencies(D)
    r = append(jb, d, f, interleaved=pairs)
    held = ref8.dequantise(codes_of(r["k_cache"]), codes_of(r["k_scales"]))
    steps = np.repeat(ref8.scale_value(codes_of(r["k_scales"])), 16, -1)[..., None] * np.ones(D)
    k, at = f64(d["k"]), 0
    for b, (t, l) in enumerate(zip(new, kv)):
        table = d["table"][b].tolist()
        y = ref.norm_rope(k[at:at + t], np.arange(l - t, l), f.numpy(), f64(d["wk"]), interleaved=pairs)
        got, s = (ref.gather(x, table, l)[l - t:] for x in (held, steps))
        z = y.reshape(t, Hkv, D // 2, 2) if pairs else y.reshape(t, Hkv, 2, D // 2).swapaxes(-1, -2)
        size = np.repeat(np.hypot(z[..., 0], z[..., 1])[..., None], 2, -1)
        size = size.reshape(y.shape) if pairs else size.swapaxes(-1, -2).reshape(y.shape)
        over = np.abs(got - y) - ref8.half_step(y / s) * s
        assert (over <= 2.5 * 2.0 ** -24 * size).all(), (b, (over / size).max() * 2 ** 24)
        at += t


def test_append_limits(jb):
    """Tokens behind max_seqlen and rows behind the last sequence are not taken."""
    new, kv = [50, 3], [70, 40]
    d = append_inputs(new, kv, 2, 2, 64, 16, BF, seed=3, behind=5)
    f = frequencies(64)
    q_out = torch.full_like(d["q"], 7.0).cuda()
    r = append(jb, d, f, max_seqlen=30, q_out=q_out)
    check_append(d, r, new, kv, f, tokens=30)
    assert (r["q"][30:50] == 7).all() and (r["q"][53:] == 7).all()


def test_append_strides_positions_and_no_norm(jb):
    """q, k and v as slices of one projection, pages and scales apart, positions of the caller's."""
    g = torch.Generator().manual_seed(4)
    n, H, Hkv, D, page = 33, 4, 2, 128, 32
    x = torch.randn(n, (H + 2 * Hkv) * D + 64, generator=g).to(BF)
    d = append_inputs([n], [90], H, Hkv, D, page, BF, seed=4)
    d["q"], d["k"], d["v"] = (x[:, a * D:(a + h) * D].view(n, h, D) for a, h in ((0, H), (H, Hkv), (H + Hkv, Hkv)))
    gpu = on_gpu(d)
    xg = x.cuda()
    q, k, v = (xg[:, a * D:(a + h) * D].view(n, h, D) for a, h in ((0, H), (H, Hkv), (H + Hkv, Hkv)))
    P = len(d["k_cache"])
    room = torch.full((2, P, Hkv * page * D + 48), 3, dtype=torch.uint8, device="cuda")
    few = torch.full((2, P, Hkv * page // 16 + 3), 9, dtype=torch.uint8, device="cuda")
    caches = [room[i, :, :Hkv * page * D].view(P, Hkv, page, D) for i in range(2)]
    scales = [few[i, :, :Hkv * page // 16].view(P, Hkv, page // 16) for i in range(2)]
    for t, name in zip(caches + scales, ("k_cache", "v_cache", "k_scales", "v_scales")):
        t.copy_(gpu[name].view(torch.uint8))
    positions = torch.arange(100000, 100000 + n, dtype=torch.int32)
    f = frequencies(D)
    args = (caches[0].view(E4M3), caches[1].view(E4M3), scales[0].view(E8M0), scales[1].view(E8M0), gpu["table"], gpu["kv"],
            f.cuda())
    r = jb.qk_norm_rope_paged8(q, k, v, *args, cu_seqlens=gpu["cu"], positions=positions.cuda(), normalize=False)
    torch.cuda.synchronize()
    assert (room[:, :, Hkv * page * D:] == 3).all() and (few[:, :, Hkv * page // 16:] == 9).all()
    eq = ref.norm_rope(f64(d["q"]), positions.numpy(), f.numpy(), normalize=False)
    tol = TURN * np.abs(eq).max(-1, keepdims=True) + 2.0 ** -8 * np.abs(eq)
    assert (np.abs(f64(r["q"]) - eq) <= tol).all()
    want = codes_of(d["v_cache"]).copy(), codes_of(d["v_scales"]).copy()
    ref8.append(*want, d["table"][0].tolist(), 90, f64(d["v"]))
    equal(codes_of(r["v_cache"].contiguous()), want[0])
    equal(codes_of(r["v_scales"].contiguous()), want[1], nan=256)
    ek = ref.norm_rope(f64(d["k"]), positions.numpy(), f.numpy(), normalize=False)
    held = ref.gather(ref8.dequantise(codes_of(r["k_cache"].contiguous()), codes_of(r["k_scales"].contiguous())),
                      d["table"][0].tolist(), 90)[90 - n:]
    assert (np.abs(held - ek) <= 2.0 ** -4 * np.abs(ek) + 2.0 ** -9 * np.abs(ek).max()).all()


# --------------------------------------------------------------- attention


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,D,H,Hkv,page,window", [
    (BF, 128, 12, 2, 64, 0), (BF, 128, 4, 4, 16, 100), (BF, 64, 8, 1, 32, 0), (BF, 64, 5, 5, 128, 33),
    (BF, 256, 4, 2, 16, 0), (BF, 256, 8, 1, 64, 70), (F32, 64, 6, 3, 16, 0), (F32, 128, 4, 1, 32, 50),
    (F32, 256, 2, 1, 16, 0),
])
def test_packed(jb, lengths, dtype, D, H, Hkv, page, window):
    new, kv = LENGTHS[lengths]
    print(f"[attn8 {lengths} {dtype} D={D} H={H}/{Hkv} page={page} window={window}]", flush=True)
    d, d8 = batch8(new, kv, H, Hkv, D, page, dtype, seed=D + H)
    strict(d, call(jb, d8, window=window), new, kv, window)


@pytest.mark.parametrize("D,H,Hkv,T", [(128, 12, 2, 1), (128, 16, 2, 3), (64, 32, 1, 1), (64, 40, 1, 1), (256, 8, 2, 1)])
@pytest.mark.parametrize("out", [BF, F32])
def test_decode(jb, D, H, Hkv, T, out):
    kv = [T, 17, 4096, 1000, 2049]
    new = [T] * 5
    d, d8 = batch8(new, kv, H, Hkv, D, 32, BF, seed=T, packed=False)
    if T == 1:
        d["q"] = d8["q"] = d["q"][:, 0]
    strict(d, call(jb, d8, out_dtype=out), new, kv)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_fp32(jb, D):
    kv = [1, 17, 3000, 513]
    d, d8 = batch8([1] * 4, kv, 8, 2, D, 16, F32, seed=D, packed=False)
    strict(d, call(jb, d8), [1] * 4, kv)


@pytest.mark.parametrize("window", [0, 1152])
def test_chunk_at_the_end_of_a_long_context(jb, window):
    new, kv = [300], [9000]
    d, d8 = batch8(new, kv, 12, 2, 128, 64, BF, seed=8)
    strict(d, call(jb, d8, window=window), new, kv, window, tokens=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_seqlen,max_kv", [(None, None), (200, 16), (200, 1 << 20)])
def test_plan_hints_change_no_result(jb, dtype, max_seqlen, max_kv):
    new, kv = [200, 1, 64], [2000, 1500, 64]
    d, d8 = batch8(new, kv, 6, 2, 64, 16, dtype, seed=3)
    d["table"] = d8["table"] = torch.cat([d["table"], torch.full((3, 200), -1, dtype=torch.int32)], 1)
    strict(d, call(jb, d8, max_seqlen=max_seqlen, max_kv=max_kv), new, kv)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_no_query_sees(jb, dtype):
    """Codes and scales that are NaN behind the rows seen, before the window and in the pages of
    nobody change no bit; pages out of range read as zeros."""
    new, kv, window = [5, 40, 1], [100, 300, 37], 90
    for w in (0, window):
        d, d8 = batch8(new, kv, 4, 2, 64, 16, dtype, seed=5)
        d["table"][1, 15] = d8["table"][1, 15] = -7  # rows 240 .. 255: zeros
        clean = call(jb, d8, window=w)
        strict(d, clean, new, kv, w)
        for x in ("k", "v"):
            c, e = d8[x + "_cache"].view(torch.uint8), d8[x + "_scales"].view(torch.uint8)
            used = set()
            for b, (t, l) in enumerate(zip(new, kv)):
                low = max(0, l - t - w + 1) if w else 0
                for j in range(d["table"].shape[1]):
                    p = int(d["table"][b, j])
                    if 0 <= p < len(c) and j * 16 < l:
                        used.add(p)
                        if j * 16 + 16 <= low:
                            c[p], e[p] = 0x7f, 255
                        elif j * 16 + 16 > l:
                            c[p, :, l - j * 16:] = 0xff
            for p in set(range(len(c))) - used:
                c[p], e[p] = 0x7f, 255
        dirty = call(jb, d8, window=w)
        assert torch.equal(clean["o"], dirty["o"]) and torch.equal(clean["lse"], dirty["lse"])


@pytest.mark.parametrize("dtype,T", [(BF, 1), (BF, 40), (F32, 1), (F32, 40)])
def test_not_finite_where_queries_see_it(jb, dtype, T):
    """A NaN code of V reaches its column of the queries that see its row, and no other."""
    kv = 200
    d, d8 = batch8([T], [kv], 4, 2, 128, 16, dtype, seed=6)
    row = 190
    p = int(d["table"][0, row // 16])
    d8["v_cache"].view(torch.uint8)[p, 1, row % 16, 77] = 0x7f
    r = call(jb, d8)
    nan = torch.isnan(r["o"].float()).cpu()
    want = torch.zeros_like(nan)
    want[max(0, row - (kv - T)):, 2:, 77] = True
    assert torch.equal(nan, want)
    assert not torch.isnan(r["lse"]).any()


def test_every_scale(jb):
    """Exponents from 20 to 234 (V, from a block to the next) and of keys that keep scores small."""
    new, kv = [1], [16 * 215]
    d, d8 = batch8(new, kv, 2, 1, 64, 16, F32, seed=7)
    codes = codes_of(d8["v_cache"]).copy()
    e = np.full((len(codes), 1, 1), 127, np.uint8)
    for j in range(215):
        e[int(d["table"][0, j])] = 20 + j
    d8["v_scales"] = torch.from_numpy(e).view(E8M0)
    # one row at a time: a window of one row
    for row in (0, 16 * 50 + 3, 16 * 107, 16 * 160 + 15, 16 * 214):
        d8["kv"] = torch.tensor([row + 1], dtype=torch.int32)
        p = int(d["table"][0, row // 16])
        want = ref8.E4M3[codes[p, 0, row % 16]] * ref8.scale_value(e[p, 0, 0])
        for q in (F32, BF):
            d8["q"] = d["q"].to(q)
            got = f64(call(jb, d8, window=1, out_dtype=F32)["o"])[0, 0]
            # One weight w, e^0 but for the rounding of the maximum that its exponent subtracts, and l = w:
            # o = fl(fl(w v) fl(1 / l)), three roundings of 2^-24; the weight's second bf16 part holds what
            # the first leaves of it (a few units of 2^-24) exactly.
            assert (np.abs(got - want) <= 2.0 ** -22 * np.abs(want)).all(), (row, q)


def test_rows_behind_the_last_sequence_stay(jb):
    new, kv = [3, 50], [10, 70]
    for dtype in (BF, F32):
        d, d8 = batch8(new, kv, 4, 2, 64, 16, dtype, behind=9)
        o = torch.full(d["q"].shape, 5.0, dtype=dtype, device="cuda")
        lse = torch.full(d["q"].shape[:-1], 5.0, device="cuda")
        r = call(jb, d8, o=o, lse=lse)
        assert (r["o"][53:] == 5).all() and (r["lse"][53:] == 5).all()
        check(d, r, new, kv)


def test_strides(jb):
    """q in a wider row, pages and scales apart."""
    new, kv, Hkv, page, D = [20, 1], [64, 50], 2, 32, 128
    d, d8 = batch8(new, kv, 4, Hkv, D, page, BF, seed=9)
    g = on_gpu(d8)
    P = len(d["k_cache"])
    wide = torch.randn(21, 6, D, device="cuda").to(BF)
    wide[:, 1:5] = g["q"]
    room = torch.zeros(2, P, Hkv * page * D + 32, dtype=torch.uint8, device="cuda")
    few = torch.full((2, P, Hkv * page // 16 + 1), 255, dtype=torch.uint8, device="cuda")
    caches = [room[i, :, :Hkv * page * D].view(P, Hkv, page, D) for i in range(2)]
    scales = [few[i, :, :Hkv * page // 16].view(P, Hkv, page // 16) for i in range(2)]
    for t, name in zip(caches + scales, ("k_cache", "v_cache", "k_scales", "v_scales")):
        t.copy_(g[name].view(torch.uint8))
    r = jb.attn_paged8(wide[:, 1:5], caches[0].view(E4M3), caches[1].view(E4M3), scales[0].view(E8M0), scales[1].view(E8M0),
                       g["table"], g["kv"], cu_seqlens=g["cu"], want_lse=True)
    torch.cuda.synchronize()
    strict(d, r, new, kv)


def test_empty_calls(jb):
    d, d8 = batch8([0, 0], [5, 0], 4, 2, 64, 16, BF)
    assert call(jb, d8)["o"].shape == (0, 4, 64)
    f = frequencies(64)
    x = append_inputs([0], [5], 4, 2, 64, 16, BF)
    before = codes_of(x["k_cache"]).copy()
    assert np.array_equal(codes_of(append(jb, x, f)["k_cache"]), before)


def test_streams_and_graphs(jb):
    """Append and attention on another stream, and captured: every replay over new inputs, with
    eager calls between the replays, gives the eager call's result."""
    new, kv = [1] * 6, [300, 5, 77, 1000, 16, 17]
    d, d8 = batch8(new, kv, 12, 2, 128, 64, BF, seed=11)
    x = append_inputs(new, kv, 12, 2, 128, 64, BF, seed=12)
    g = on_gpu({**d8, **{n: x[n] for n in ("q", "k", "v", "wq", "wk")}})
    f = frequencies(128).cuda()
    fresh = [t.clone() for t in (g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"])]

    def step(c):
        a = jb.qk_norm_rope_paged8(g["q"], g["k"], g["v"], *c, g["table"], g["kv"], f, g["wq"], g["wk"], cu_seqlens=g["cu"])
        return jb.attn_paged8(a["q"], *c, g["table"], g["kv"], cu_seqlens=g["cu"], max_seqlen=1, want_lse=True)

    def reset(c):
        for t, s in zip(c, fresh):
            t.view(torch.uint8).copy_(s.view(torch.uint8))

    own, theirs = ([t.clone() for t in fresh] for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(own)
        reset(own)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(own)
    for k in range(4):
        g["q"].copy_(torch.randn(g["q"].shape, generator=torch.Generator().manual_seed(k)).to(BF))
        g["k"].copy_(torch.randn(g["k"].shape, generator=torch.Generator().manual_seed(9 + k)).to(BF))
        reset(own)
        reset(theirs)
        graph.replay()
        want = step(theirs)
        torch.cuda.synchronize()
        assert torch.equal(out["o"], want["o"]) and torch.equal(out["lse"], want["lse"])
        for a, b in zip(own, theirs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_cache_past_32_bit_offsets(jb):
    """Pages and scales more than 2^32 bytes apart from the pool's start: append, then attention."""
    new, kv, H, Hkv, D, page = [3, 1], [40, 600], 4, 2, 64, 16
    x = append_inputs(new, kv, H, Hkv, D, page, BF, seed=40)
    P, far = len(x["k_cache"]), 1 << 27
    pools = [torch.empty(P * far, dtype=torch.uint8, device="cuda") for _ in range(2)]
    caches = [p.as_strided((P, Hkv, page, D), (far, page * D, D, 1)) for p in pools]
    scales = [p.as_strided((P, Hkv, page // 16), (far, page // 16, 1), 1 << 26) for p in pools]
    assert P * far > 1 << 32
    for t, name in zip(caches + scales, ("k_cache", "v_cache", "k_scales", "v_scales")):
        t.copy_(x[name].view(torch.uint8))
    g = on_gpu({n: x[n] for n in ("q", "k", "v", "wq", "wk", "table", "kv", "cu")})
    f = frequencies(D)
    views = (caches[0].view(E4M3), caches[1].view(E4M3), scales[0].view(E8M0), scales[1].view(E8M0))
    r = jb.qk_norm_rope_paged8(g["q"], g["k"], g["v"], *views, g["table"], g["kv"], f.cuda(), g["wq"], g["wk"],
                               cu_seqlens=g["cu"])
    torch.cuda.synchronize()
    check_append(x, {n: t if n == "q" else t.view(torch.uint8).contiguous().view(t.dtype) for n, t in r.items()}, new, kv, f)
    o = jb.attn_paged8(r["q"], *views, g["table"], g["kv"], cu_seqlens=g["cu"], want_lse=True)
    torch.cuda.synchronize()
    held = dict(x, q=r["q"].cpu(), k_cache=torch.from_numpy(ref8.dequantise(*(codes_of(t.contiguous()) for t in (caches[0], scales[0])))),
                v_cache=torch.from_numpy(ref8.dequantise(*(codes_of(t.contiguous()) for t in (caches[1], scales[1])))))
    strict(held, o, new, kv)


@pytest.mark.parametrize("G", [1, 3, 8, 9, 16, 17, 32])
def test_every_width_of_the_decode_kernels(jb, G):
    """Queries to a key head on both sides of 8, 16 and 32 columns, windows and single rows too."""
    kv = [1, 40, 333, 2000]
    for T, window in ((1, 0), (1, 50), (2, 0)):
        d, d8 = batch8([T] * 4, kv, 2 * G, 2, 128, 16, BF, seed=G + T, packed=False)
        for out in (BF, F32):
            strict(d, call(jb, d8, window=window, out_dtype=out), [T] * 4, kv, window)


def test_a_second_stream_and_workspaces_of_their_own(jb):
    """Two calls that run at the same time, each on a stream of its own."""
    d, d8 = batch8([1] * 4, [3000, 5, 800, 64], 12, 2, 128, 64, BF, seed=50, packed=False)
    g = on_gpu(d8)
    args = (g["q"][:, 0], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"])
    want = jb.attn_paged8(*args)["o"]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [jb.attn_paged8(*args, stream=s if i else s.cuda_stream)["o"] for i, s in enumerate(streams) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in got)
