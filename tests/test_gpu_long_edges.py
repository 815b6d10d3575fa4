"""GPU tests of the long-context operators (a cache in 8 bits, selected pages) at the edges that the
parity tests (test_gpu_attn8, test_gpu_blocks) do not reach."""
import numpy as np
import pytest
import torch

from oracle import blocks as ref8
from test_gpu_attn import BF, F32
from test_gpu_attn8 import E4M3, E8M0, jb  # noqa: F401

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
