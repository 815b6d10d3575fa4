"""GPU tests of the long-context operators (a cache in 8 bits, selected pages) at the edges that the
parity tests (test_gpu_attn8, test_gpu_blocks) do not reach."""
import numpy as np
import pytest
import torch

from oracle import blocks as ref8
from test_gpu_attn import BF, F32, f64
from test_gpu_attn8 import E4M3, E8M0, codes_of, equal, frequencies, jb  # noqa: F401

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
