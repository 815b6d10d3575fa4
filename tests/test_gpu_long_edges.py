"""GPU tests of the long-context operators (a cache in 8 bits, selected pages) at the edges that the
parity tests (test_gpu_attn8, test_gpu_blocks) do not reach: values at the end of the range, dense
appends, keys with positions of the caller's and without the norm, lists long enough to be cut into
pieces, workgroups that score several tiles of tokens, malformed offsets and lengths.

Bounds are those of the parity tests, and a key's that of test_append_codes_at_their_borders: its code
is that of its value in 64 bits but where that lies within 2.5 * 2^-24 hypot(a, b) of a border, a and b the
members of its pair; where positions reach p, its angles (products of a position and a frequency of at most
1, rounded in 64 bits, on either side) differ by at most p 2^-51."""
import numpy as np
import pytest
import torch

from layer_checks import same_kind
from oracle import attention as ref
from oracle import blocks as ref8
from test_gpu_attn import BF, F32, f64
from test_gpu_attn8 import (E4M3, E8M0, append, append_inputs, batch8, check_append, codes_of, equal, frequencies, jb,  # noqa: F401
                            on_gpu, strict)
from test_gpu_blocks import CACHES, attend, check_blocks, inputs, places, some_lists

pytestmark = pytest.mark.gpu

# ------------------------------------------- codes whose value passes the range


def past_the_range(T, H, Hkv, D, dtype, window):
    """A sequence of 100 rows, T new ones, with one row of V that some of them see and some do not (the
    last one, or the first of the first token's window), in a block of zeros under a scale of its own:
    (the call's tensors, that row, which tokens see it)."""
    page, kv = 16, 100
    g = torch.Generator().manual_seed(D + T + H)
    P = -(-kv // page) + 1
    codes = [torch.randint(0, 256, (P, Hkv, page, D), generator=g).to(torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 0
    scales = [torch.full((P, Hkv, 1), 118, dtype=torch.uint8) for _ in range(2)]
    row = kv - T - window + 1 if window else kv - 1
    seen = torch.tensor([i == (0 if window else T - 1) for i in range(T)])
    codes[1][row // page] = 0
    q = torch.randn(T, H, D, generator=g).to(dtype)
    table = torch.arange(P - 1, dtype=torch.int32).view(1, -1)
    return dict(q=q.cuda(), codes=codes, scales=scales, table=table.cuda(), kv=torch.tensor([kv], dtype=torch.int32).cuda(),
                cu=torch.tensor([0, T], dtype=torch.int32).cuda(), window=window), row, seen


def outputs(jb, d, lists, out):
    (k, v), (ks, vs) = ([t.clone().cuda() for t in d[n]] for n in ("codes", "scales"))
    caches, scales = (k.view(E4M3), v.view(E4M3)), (ks.view(E8M0), vs.view(E8M0))
    if lists is None:
        r = jb.attn_paged8(d["q"], *caches, *scales, d["table"], d["kv"], cu_seqlens=d["cu"], window=d["window"],
                           out_dtype=out, want_lse=True)
    else:
        r = jb.attn_blocks(d["q"], *caches, d["table"], d["kv"], lists.cuda(), k_scales=scales[0], v_scales=scales[1],
                           cu_seqlens=d["cu"], out_dtype=out, want_lse=True)
    torch.cuda.synchronize()
    return r["o"].float().cpu(), r["lse"].cpu()


@pytest.mark.parametrize("dtype,D,T,H,Hkv", [
    (BF, 64, 2, 4, 2), (BF, 128, 3, 4, 2), (BF, 256, 2, 8, 2), (BF, 128, 2, 10, 1), (BF, 64, 3, 8, 2), (BF, 256, 2, 24, 1),
    (BF, 128, 4, 36, 2), (F32, 64, 3, 4, 2), (F32, 128, 5, 40, 2),
])
@pytest.mark.parametrize("form", ["causal", "window", "lists"])
def test_values_past_the_range(jb, dtype, D, T, H, Hkv, form):
    """A code whose value is 2^128 or more reads as an infinity and has no part in the tokens that do
    not see its row: their outputs keep every bit.  The code below it is a number like any other."""
    print(f"[past the range {form} {dtype} D={D} T={T} H={H}/{Hkv}]", flush=True)
    d, row, seen = past_the_range(T, H, Hkv, D, dtype, 40 if form == "window" else 0)
    page = row // 16
    lists = None
    if form == "lists":
        lists = torch.full((T, Hkv, 4), -1, dtype=torch.int32)
        lists[:, :, 0], lists[:, :, 1], lists[:, :, 2] = 1, 2, page
    for out in (F32, BF):
        clean = outputs(jb, d, lists, out)
        assert torch.isfinite(clean[0]).all()
        for e, codes in ((247, (0x78, 0xf8, 0x7e)), (250, (0x60,)), (254, (0x40, 0xc1)), (255, (0,))):
            for code in codes:
                d["scales"][1][page] = e
                d["codes"][1][page, :, row % 16, 5] = code
                o, lse = outputs(jb, d, lists, out)
                assert torch.equal(lse, clean[1])
                if e == 255:  # (every value of the 16 rows is NaN: tokens that see another of them too)
                    others = torch.arange(T) < T - 1 - row % 16 if not d["window"] else torch.arange(T) >= 16 - row % 16
                    assert torch.equal(o[others], clean[0][others]) and torch.isnan(o[seen]).all()
                    continue
                assert torch.equal(o[~seen], clean[0][~seen]), (e, code)
                assert not torch.isfinite(o[seen][..., 5]).any(), (e, code)
                rest = torch.arange(D) != 5
                assert torch.equal(o[seen][..., rest], clean[0][seen][..., rest]), (e, code)
                # The largest value that is a number, 1.875 * 2^127.  Its weight is e^(x - m) with an m
                # that may lag 2^8 behind, so the sum before the division by l may pass the range; where
                # all scores are 0 every weight is 1 and the sum is the value.
                d["codes"][1][page, :, row % 16, 5] = (code & 0x78) - 1
                o = outputs(jb, d, lists, out)[0]
                assert torch.equal(o[~seen], clean[0][~seen]), (e, code)
                assert (o[seen][..., 5] > 2.0 ** 100).all()
                o = outputs(jb, dict(d, q=torch.zeros_like(d["q"])), lists, out)[0]
                assert torch.isfinite(o).all() and (o[seen][..., 5] > 2.0 ** 120).all(), (e, code)
                d["codes"][1][page, :, row % 16, 5] = 0
            d["scales"][1][page] = 118


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_values_stay_numbers(jb, dtype):
    """The largest finite keys and values of each type, and those around the last codes' borders, are
    appended as codes that stand for finite values: of 1.9375 * 2^127 and more the nearest code's value
    would be 2^128.  In rows of their own, and in 16 rows whose scale in the cache is larger."""
    H, Hkv, D, page, kv = 2, 1, 64, 16, 40
    top = torch.finfo(dtype).max
    sizes = [top, 1.9375 * 2.0 ** 127, 1.9296875 * 2.0 ** 127, 1.875 * 2.0 ** 127, 1.75 * 2.0 ** 127, 2.0 ** 127, 3.0, float("inf")]
    n = 30  # rows 10 .. 39: 6 of the first 16 share them with rows before, whose scale is 2^123
    x = torch.tensor(sizes, dtype=torch.float64).to(dtype).repeat(n * D // 8 + 1)[:n * D].view(n, 1, D)
    x = torch.where(torch.arange(D) % 3 == 0, -x, x)
    q = torch.zeros(n, H, D, dtype=dtype)
    cu, lens = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([kv], dtype=torch.int32).cuda()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    caches = [torch.zeros(3, Hkv, page, D, dtype=torch.uint8).cuda().view(E4M3) for _ in range(2)]
    scales = [torch.full((3, Hkv, 1), 250, dtype=torch.uint8).cuda().view(E8M0) for _ in range(2)]
    r = jb.qk_norm_rope_paged8(q.cuda(), x.cuda(), x.cuda(), *caches, *scales, table.cuda(), lens, frequencies(D).cuda(),
                               cu_seqlens=cu, positions=torch.zeros(n, dtype=torch.int32).cuda(), normalize=False)
    torch.cuda.synchronize()
    want = np.zeros((3, Hkv, page, D), np.uint8), np.full((3, Hkv, 1), 250, np.uint8)
    ref8.append(*want, table[0].tolist(), kv, f64(x))
    assert want[1].ravel().tolist() == [247, 247, 250]
    for c, s in zip(caches, scales):
        equal(codes_of(c), want[0])
        equal(codes_of(s), want[1], nan=256)
        held = ref8.dequantise(codes_of(c), codes_of(s))
        held = np.concatenate([held[p, 0] for p in (2, 0, 1)])[10:kv]
        fine = np.isfinite(f64(x)[:, 0])
        assert np.isnan(held[~fine]).all() and (np.abs(held[fine]) < 2.0 ** 128).all()
        # half a step is at most 2^-4 of a value (and 2^-10 of the largest scale, 2^123), the next code
        # down from 2^128 a whole one: 2^-4 of it
        assert (np.abs(held - f64(x)[:, 0])[fine] <= 2.0 ** -4 * np.abs(f64(x)[:, 0][fine]) + 2.0 ** 113).all()
    assert r["k_cache"] is caches[0]


# ------------------------------------------------------------------ the append


def check_keys(d, r, new, kv, f, pairs=False, normalize=True, positions=None):
    """The codes of the appended keys against their values in 64 bits."""
    D = d["k"].shape[-1]
    k, Hkv = f64(d["k"]).reshape(-1, *d["k"].shape[-2:]), d["k"].shape[-2]
    held = ref8.dequantise(codes_of(r["k_cache"]), codes_of(r["k_scales"]))
    steps = np.repeat(ref8.scale_value(codes_of(r["k_scales"])), 16, -1)[..., None] * np.ones(D)
    at, rot = 0, 2 * len(f)
    for b, (t, l) in enumerate(zip(new, kv)):
        table, skip = d["table"][b].tolist(), max(0, t - l)  # (tokens without a row)
        place = np.arange(l - t, l) if positions is None else f64(positions)[at:at + t]
        y = ref.norm_rope(k[at:at + t], place, f.numpy(), f64(d["wk"]) if normalize else None, interleaved=pairs,
                          normalize=normalize)[skip:]
        got, s = (ref.gather(x, table, l)[l - t + skip:] for x in (held, steps))
        size = np.abs(y)  # (values that are not rotated: one rounding)
        z = y[..., :rot].reshape(*y.shape[:2], rot // 2, 2) if pairs else \
            y[..., :rot].reshape(*y.shape[:2], 2, rot // 2).swapaxes(-1, -2)
        z = np.repeat(np.hypot(z[..., 0], z[..., 1])[..., None], 2, -1)
        size[..., :rot] = z.reshape(*y.shape[:2], rot) if pairs else z.swapaxes(-1, -2).reshape(*y.shape[:2], rot)
        with np.errstate(invalid="ignore", divide="ignore"):
            over = np.abs(got - y) - ref8.half_step(y / s) * s
        over[s == 0] = -1  # (a page out of range)
        assert (over <= (2.5 * 2.0 ** -24 + np.abs(place).max(initial=0) * 2.0 ** -51) * size).all(), \
            (b, (over / np.maximum(size, 1e-300)).max() * 2 ** 24)
        at += t


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33])
@pytest.mark.parametrize("dtype,D,H,Hkv,page,pairs", [(BF, 128, 6, 2, 64, False), (F32, 64, 2, 2, 16, True), (BF, 256, 4, 1, 32, False)])
def test_dense_append(jb, T, dtype, D, H, Hkv, page, pairs):
    """[B, T, H, D] (and [B, H, D]) without offsets: first rows at every place of 16, sequences with
    fewer rows than new tokens, and none."""
    print(f"[dense append8 T={T} {dtype} D={D} H={H}/{Hkv} page={page}]", flush=True)
    new = [T] * 18
    kv = [T + 16 * (b % 3) + b for b in range(16)] + [T - 1, 0]
    f = frequencies(D)
    d = append_inputs(new, kv, H, Hkv, D, page, dtype, seed=T + D)
    d["table"][4, 0] = 1 << 20  # (no page: rows that are not stored)
    for name, heads in (("q", H), ("k", Hkv), ("v", Hkv)):
        d[name] = d[name].view(18, T, heads, D)
    d["cu"] = None
    r = append(jb, d, f, interleaved=pairs)
    assert r["q"].shape == (18, T, H, D)
    check_append(d, r, new, kv, f, pairs)
    check_keys(d, r, new, kv, f, pairs)
    packed = append(jb, dict(d, **{n: d[n].flatten(0, 1) for n in "qkv"}, cu=torch.arange(19, dtype=torch.int32) * T), f,
                    interleaved=pairs)
    same = lambda x: all(torch.equal(r[n].flatten().view(torch.uint8), x[n].flatten().view(torch.uint8)) for n in r)  # noqa: E731
    assert same(packed)
    if T == 1:
        d1 = dict(d, **{n: d[n][:, 0] for n in "qkv"})
        assert append(jb, d1, f, interleaved=pairs)["q"].shape == (18, H, D)
        assert same(append(jb, d1, f, interleaved=pairs))


@pytest.mark.parametrize("normalize,far", [(True, True), (False, True), (False, False)])
@pytest.mark.parametrize("dtype,D,rot,pairs", [(BF, 128, 128, False), (BF, 64, 32, True), (F32, 128, 64, False), (F32, 256, 256, True)])
def test_keys_at_their_borders(jb, dtype, D, rot, pairs, normalize, far):
    """Positions of the caller's (up to a million) and keys without the norm, heads rotated in part."""
    new, kv = [200, 1, 333], [203, 90, 400]
    d = append_inputs(new, kv, 2, 2, D, 32, dtype, seed=D + rot)
    f = frequencies(rot)
    positions = torch.randint(0, 10 ** 6, (sum(new),), generator=torch.Generator().manual_seed(1), dtype=torch.int32) if far else None
    if not normalize:
        d = dict(d, wq=torch.empty(0), wk=torch.empty(0))
    g = on_gpu(d)
    w = (g["wq"], g["wk"]) if normalize else ()
    r = jb.qk_norm_rope_paged8(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"],
                               g["kv"], f.cuda(), *w, cu_seqlens=g["cu"], interleaved=pairs, normalize=normalize,
                               positions=None if positions is None else positions.cuda())
    torch.cuda.synchronize()
    check_keys(d, r, new, kv, f, pairs, normalize, positions)


# ------------------------------------------------------- lists cut into pieces

# bits, D, query heads, key heads, page, entries of a list: about 20 steps of the workgroup
CUT = [(8, 64, 6, 2, 64, 40), (8, 128, 12, 2, 64, 40), (8, 128, 12, 1, 128, 20), (8, 256, 4, 2, 32, 40), (8, 64, 20, 1, 64, 40),
       (16, 64, 2, 2, 128, 40), (16, 128, 12, 2, 128, 40), (16, 256, 4, 1, 64, 40)]


def long_lists(new, kv, Hkv, page, count, seed):
    """Lists of every length, the first and the last token's full."""
    lists = some_lists(new, kv, Hkv, page, count, seed)
    g = np.random.default_rng(seed + 1)
    at = list(places(new, kv))
    for t, b, p in (max(at, key=lambda x: x[2]), at[0]):
        own = p // page
        for h in range(Hkv if p >= 0 else 0):
            n = min(count, own + 1)
            lists[t, h] = -1
            lists[t, h, :n] = torch.from_numpy(np.sort(g.choice(own + 1, n, replace=False)).astype(np.int32))
    return lists


def pieces(jb, B, T, n, bits, D, H, Hkv, page, count, pages, packed):
    """Pieces that a unit's lists are cut into, from the workspace: (D + 2) floats a row and piece."""
    shape = jb.AttnShape(B, T, H, Hkv, D, 0, page, pages, 4096, 0, 0, jb.JB_BF16, jb.JB_BF16, jb.CACHE_E4M3 if bits == 8 else 0,
                         0, 0, 0, 0)
    return max(1, jb.attn_blocks_workspace_size(shape, n, packed, count) // (n * H * (D + 2) * 4))


@pytest.mark.parametrize("case", CUT)
@pytest.mark.parametrize("out", [BF, F32])
def test_decode_over_lists_in_pieces(jb, case, out):
    """A decode step whose lists are cut: sequences that fill them, with a page or two, without rows."""
    bits, D, H, Hkv, page, count = case
    print(f"[decode in pieces {case}]", flush=True)
    kv = [count * page + 77, 1, 100, 0, 2 * count * page // 3, page * 2]
    new = [1] * 6
    d, g = inputs(new, kv, H, Hkv, D, page, BF, bits, seed=D, packed=False)
    assert pieces(jb, 6, 1, 6, *case, d["table"].shape[1], False) > 1
    g["q"] = g["q"][:, 0].contiguous()
    lists = long_lists(new, kv, Hkv, page, count, D)
    check_blocks(d, attend(jb, g, lists, out_dtype=out), lists, new, kv)


@pytest.mark.parametrize("case", CUT)
@pytest.mark.parametrize("limit", [None, 4])
def test_packed_lists_in_pieces(jb, case, limit):
    """Neighbouring tokens' lists merged and cut; tokens of nobody, and those behind max_seqlen, stay."""
    bits, D, H, Hkv, page, count = case
    print(f"[packed in pieces {case} {limit}]", flush=True)
    new, kv = [3, 1, 0, 6, 4], [count * page + 77, 300, 9, 2 * page, 2]
    n, behind = sum(new), 3
    d, g = inputs(new, kv, H, Hkv, D, page, BF, bits, seed=D + 1, behind=behind)
    T = n + behind if limit is None else limit
    assert pieces(jb, 5, T, n + behind, *case, d["table"].shape[1], True) > 1
    lists = long_lists(new, kv, Hkv, page, count, D)
    lists = torch.cat([lists, torch.zeros(behind, Hkv, count, dtype=torch.int32)])
    o = torch.full((n + behind, H, D), 5.0, dtype=BF, device="cuda")
    lse = torch.full((n + behind, H), 5.0, device="cuda")
    r = attend(jb, g, lists, max_seqlen=limit, o=o, lse=lse)
    stay = [*range(n, n + behind)] + ([8, 9] if limit else [])
    assert (r["o"][stay] == 5).all() and (r["lse"][stay] == 5).all()
    check_blocks(d, r, lists, new, kv, tokens=limit)


@pytest.mark.parametrize("case", CUT)
def test_dense_lists_in_pieces(jb, case):
    bits, D, H, Hkv, page, count = case
    T, kv = 3, [count * page + 200, 2]
    d, g = inputs([T] * 2, kv, H, Hkv, D, page, BF, bits, seed=D + 2, packed=False)
    assert pieces(jb, 2, T, 2 * T, *case, d["table"].shape[1], False) > 1
    lists = long_lists([T] * 2, kv, Hkv, page, count, D)
    check_blocks(d, attend(jb, g, lists.view(2, T, Hkv, count), out_dtype=F32), lists, [T] * 2, kv)


@pytest.mark.parametrize("case", CUT)
def test_not_finite_in_a_piece(jb, case):
    """A value that is not finite, in a page that one of three merged tokens lists, is in one piece of
    the unit: it reaches that token and changes no bit of the others."""
    bits, D, H, Hkv, page, count = case
    T, kv = 3, count * page + page
    d, g = inputs([T], [kv], H, Hkv, D, page, BF, bits, seed=D + 3)
    assert pieces(jb, 1, T, T, *case, d["table"].shape[1], True) > 1
    lists = torch.arange(count, dtype=torch.int32).expand(T, Hkv, count).contiguous()
    lists[0] = torch.where(lists[0] >= count // 2, lists[0] + 1, lists[0])  # all but page count / 2
    lists[2] = lists[0]
    clean = attend(jb, g, lists)
    check_blocks(d, clean, lists, [T], [kv])
    v = g["v_cache"].view(torch.uint8) if bits == 8 else g["v_cache"]
    v[int(d["table"][0, count // 2]), Hkv - 1, 5, 9] = 0x7f if bits == 8 else float("inf")
    r = attend(jb, g, lists)
    want = torch.zeros(T, H, D, dtype=torch.bool)
    want[1, H - H // Hkv:, 9] = True
    assert torch.equal(~torch.isfinite(r["o"].float()).cpu(), want)
    assert torch.equal(r["o"].cpu()[~want], clean["o"].cpu()[~want]) and torch.equal(r["lse"], clean["lse"])


# ----------------------------------------------- several tiles of a workgroup


@pytest.mark.parametrize("dtype,D,H,Hkv,bits,packed", [
    (BF, 128, 8, 4, 16, True), (BF, 64, 5, 5, 8, True), (BF, 256, 4, 4, 16, True), (BF, 128, 6, 3, 8, False), (BF, 256, 6, 3, 8, False),
    (F32, 64, 4, 2, 32, True),
])
def test_scores_of_many_tiles(jb, dtype, D, H, Hkv, bits, packed):
    """So many tiles of 32 tokens that a workgroup takes several in turn, and keeps the means of their
    pages: sequences end inside its tiles, some have no tokens or no rows, tables are wider than any
    sequence."""
    page, width = 16, 1020
    if packed:
        new = [700, 0, 33, 500, 1, 64, 300, 0, 450, 31, 5]
        kv = [16000, 5, 40, 700, 900, 64, 250, 0, 9000, 31, 8000]
    else:
        new, kv = [410] * 5, [410, 16300, 0, 5000, 411]
    print(f"[scores of many tiles {dtype} D={D} H={H}/{Hkv} {bits} packed={packed}]", flush=True)
    behind = 3 if packed else 0
    d, g = inputs(new, kv, H, Hkv, D, page, dtype, bits, seed=D + H, packed=packed, behind=behind)
    n, P, G = sum(new), len(d["k_cache"]), H // Hkv
    slots = n // 32 + len(new) if packed else len(new) * -(-new[0] // 32)
    assert dtype == F32 or slots * Hkv * 8 >= 2 * (256 if D == 256 else 512)  # (two tiles a workgroup and more)
    wide = torch.full((len(new), width), -1, dtype=torch.int32)
    wide[:, :d["table"].shape[1]] = d["table"]
    before = torch.randn(P, Hkv, D, generator=torch.Generator().manual_seed(1))
    out = torch.full((n + behind, Hkv, width), 5.0, device="cuda")
    means = before.cuda()
    q = g["q"]
    jb.block_scores(q, g["k_cache"], means, wide.cuda(), g["kv"], k_scales=g["k_scales"], cu_seqlens=g["cu"],
                    scores=out if packed else out.view(*q.shape[:2], Hkv, width))
    torch.cuda.synchronize()
    k, q = f64(d["k_cache"]), f64(d["q"]).reshape(-1, H, D)
    want_m, tol = f64(before), np.zeros((P, Hkv, D))
    for b, (t, l) in enumerate(zip(new, kv)):
        for j in range(max(0, l - t) // page, -(-l // page) if t else 0):
            p, rows = int(d["table"][b, j]), min(page, l - j * page)
            want_m[p], mag = ref8.mean_of(k[p, :, :rows].swapaxes(0, 1))
            tol[p] = (rows + 1) * 2.0 ** -24 * mag
    got_m = same_kind(means, want_m)
    assert (np.abs(got_m - want_m) <= tol).all()
    want = np.full((n + behind, Hkv, width), 5.0)
    slack, at = np.zeros_like(want), 0
    for b, (t, l) in enumerate(zip(new, kv)):
        own = np.arange(l - t, l) // page
        seen = np.arange(width)[None] <= own[:, None]
        pages = -(-l // page)
        for h in range(Hkv):
            m, qs = got_m[d["table"][b, :pages].numpy(), h], q[at:at + t, h * G:(h + 1) * G]
            x = np.full((t, width), -np.inf)
            if t and pages:
                x[:, :pages] = ref8.scores(qs, m)
                slack[at:at + t, h, :pages] = (3 * D + 2) * 2.0 ** -24 * ref8.scores(np.abs(qs), np.abs(m))
            want[at:at + t, h] = np.where(seen, x, -np.inf)
        at += t
    got = same_kind(out, want)
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= slack[fine]).all()


# ------------------------------------------------------------- dense batches


@pytest.mark.parametrize("dtype,D,T", [(BF, 128, 40), (BF, 64, 130), (F32, 64, 20), (BF, 256, 12)])
def test_dense_chunks(jb, dtype, D, T):
    """Attention in 8 bits of [B, T, H, D], more than 32 queries to a key head."""
    new, kv = [T] * 3, [T + 200, T, T - 5]
    d, d8 = batch8(new, kv, 8, 2, D, 32, dtype, seed=T, packed=False)
    g = on_gpu(d8)
    r = jb.attn_paged8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"], want_lse=True)
    torch.cuda.synchronize()
    strict(d, r, new, kv)


@pytest.mark.parametrize("width", [20, 300, 1500])
def test_select_of_a_dense_batch(jb, width):
    """[B, T, Hkv, max_pages]: one wave a row, and four."""
    B, T, Hkv, page, count = 3, 5, 2, 16, 9
    x = torch.randn(B, T, Hkv, width, generator=torch.Generator().manual_seed(width))
    kv = [width * page, 3, width * page // 2 + 1]
    got = jb.block_select(x.cuda(), torch.tensor(kv, dtype=torch.int32).cuda(), count, page, first=2, recent=2).cpu()
    assert got.shape == (B, T, Hkv, count)
    for t, b, p in places([T] * B, kv):
        for h in range(Hkv):
            want = ref8.select(x.view(-1, Hkv, width)[t, h].tolist(), p // page, count, 2, 2) if p >= 0 else [-1] * count
            assert got.view(-1, Hkv, count)[t, h].tolist() == want, (t, h)


# ------------------------------------------------- malformed offsets and lengths


def guarded(shape, dtype, fill):
    """A tensor on the GPU with as many rows before and behind it, all of one value, and the check of those."""
    n = shape[0]
    t = torch.full((3 * n, *shape[1:]), fill, dtype=dtype, device="cuda")
    return t[n:2 * n], lambda: (t[:n] == fill).all() and (t[2 * n:] == fill).all()


@pytest.mark.parametrize("dtype,bits", CACHES)
@pytest.mark.parametrize("cu", [[0, 500, -40, 120], [120, 80, 40, 0], [-10 ** 9, 10 ** 9, 7, 9], [130, 140, 150, 160]])
def test_malformed_offsets_stay_in_bounds(jb, dtype, bits, cu):
    """Offsets past the rows, negative and decreasing ones, lengths past the table and negative: some
    rows are wrong, but nothing outside the tensors is written."""
    print(f"[malformed {dtype} {bits} {cu}]", flush=True)
    n, H, Hkv, D, page, count = 120, 4, 2, 64, 16, 3
    d, g = inputs([40] * 3, [60] * 3, H, Hkv, D, page, dtype, bits, seed=7)
    for kv in ([10 ** 9, -5, 64], [60, 60, 60], [-2 ** 31, 2 ** 31 - 1, 1]):
        g["cu"], g["kv"] = torch.tensor(cu, dtype=torch.int32).cuda(), torch.tensor(kv, dtype=torch.int32).cuda()
        P, width = len(d["k_cache"]), d["table"].shape[1]
        checks = []

        def out(shape, dt=torch.float32, fill=7):
            t, check = guarded(shape, dt, fill)
            checks.append(check)
            return t

        if bits == 8:
            x = append_inputs([40] * 3, [60] * 3, H, Hkv, D, page, dtype, seed=8)
            codes = [out((P, Hkv, page, D), torch.uint8).view(E4M3) for _ in range(2)]
            scales = [out((P, Hkv, page // 16), torch.uint8, 120).view(E8M0) for _ in range(2)]
            jb.qk_norm_rope_paged8(*(x[c].cuda() for c in "qkv"), *codes, *scales, g["table"], g["kv"], frequencies(D).cuda(),
                                   cu_seqlens=g["cu"], q_out=out((n, H, D), dtype))
            jb.attn_paged8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"],
                           cu_seqlens=g["cu"], o=out((n, H, D), dtype), lse=out((n, H)))
            jb.attn_paged8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"],
                           cu_seqlens=g["cu"], max_seqlen=1, o=out((n, H, D), dtype), lse=out((n, H)))
        scores = jb.block_scores(g["q"], g["k_cache"], out((P, Hkv, D)), g["table"], g["kv"], k_scales=g["k_scales"],
                                 cu_seqlens=g["cu"], scores=out((n, Hkv, width)))["scores"]
        jb.block_select(scores, g["kv"], count, page, cu_seqlens=g["cu"], blocks=out((n, Hkv, count), torch.int32))
        lists = torch.arange(count, dtype=torch.int32).expand(n, Hkv, count).contiguous()
        attend(jb, g, lists, o=out((n, H, D), dtype), lse=out((n, H)))
        torch.cuda.synchronize()
        assert all(c() for c in checks)


@pytest.mark.parametrize("dtype,bits", CACHES)
def test_lengths_past_the_table(jb, dtype, bits):
    """Lengths are taken as in [0, max_pages * page]: outputs and caches are those of such lengths."""
    new, H, Hkv, D, page, count = [5, 1, 20, 3], 4, 2, 64, 16, 3
    d, g = inputs(new, [160] * 4, H, Hkv, D, page, dtype, bits, seed=9)
    x = append_inputs(new, [160] * 4, H, Hkv, D, page, dtype, seed=10)
    means = torch.from_numpy(f64(d["k_cache"]).mean(2)).float()
    lists = torch.tensor([0, 4, 9], dtype=torch.int32).expand(sum(new), Hkv, count).contiguous()
    got = []
    for kv in ([161, -1, 2 ** 31 - 1, -2 ** 31], [160, 0, 160, 0]):
        g["kv"] = torch.tensor(kv, dtype=torch.int32).cuda()
        y = []
        if bits == 8:
            a = append(jb, dict(x, kv=g["kv"].cpu(), table=d["table"]), frequencies(D))
            y += [a[c] for c in ("q", "k_cache", "v_cache", "k_scales", "v_scales")]
            r = jb.attn_paged8(g["q"], g["k_cache"], g["v_cache"], g["k_scales"], g["v_scales"], g["table"], g["kv"],
                               cu_seqlens=g["cu"], want_lse=True)
            y += [r["o"], r["lse"]]
        s = jb.block_scores(g["q"], g["k_cache"], means.cuda(), g["table"], g["kv"], k_scales=g["k_scales"], cu_seqlens=g["cu"])
        y += [s["scores"], s["means"], jb.block_select(s["scores"], g["kv"], count, page, cu_seqlens=g["cu"])]
        r = attend(jb, g, lists)
        y += [r["o"], r["lse"]]
        got.append([t.contiguous().view(torch.uint8).clone() for t in y])
    assert all(torch.equal(a, b) for a, b in zip(*got))
