"""CPU tests around the attention-layer operators: the comparisons of their GPU tests and the
binding's and the library's handling of calls at their limits."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as ref


def test_comparisons_refuse_nan():
    """An output of NaN passes neither comparison of the strict run of the GPU tests; the right one
    passes both."""
    import test_gpu_attn
    import test_gpu_rope
    from test_gpu_layer_strict import strict
    check, near = strict(test_gpu_attn.check, test_gpu_rope.near)
    new, kv, H, Hkv, D, page = [3, 1], [20, 7], 2, 1, 64, 16
    d = test_gpu_attn.batch(new, kv, H, Hkv, D, page, torch.float32)
    o, lse = [], []
    at = 0
    for b, (t, l) in enumerate(zip(new, kv)):
        k, v = (ref.gather(d[c].numpy().astype(np.float64), d["table"][b].tolist(), l) for c in ("k_cache", "v_cache"))
        eo, el, _, _ = ref.attend(d["q"][at:at + t].numpy(), k, v)
        o.append(eo), lse.append(el)
        at += t
    o, lse = (torch.tensor(np.concatenate(x), dtype=torch.float32) for x in (o, lse))
    check(d, dict(o=o, lse=lse), new, kv)
    for name, i in (("o", (0, 1, 5)), ("o", (3, 0, 63)), ("lse", (2, 1))):
        r = dict(o=o.clone(), lse=lse.clone())
        r[name][i] = float("nan")
        with pytest.raises(AssertionError):
            check(d, r, new, kv)
    # rows behind the last sequence are nobody's
    r = dict(o=torch.cat([o, o[:1] * float("nan")]), lse=torch.cat([lse, lse[:1] * float("nan")]))
    check(dict(d, q=torch.cat([d["q"], d["q"][:1]])), r, new, kv)
    want = np.ones((2, 3, 4))
    near(torch.ones(2, 3, 4), want, want)
    for bad in (torch.full((2, 3, 4), float("nan")), torch.tensor([1.0] * 23 + [float("nan")]).view(2, 3, 4)):
        with pytest.raises(AssertionError):
            near(bad, want, want)


@pytest.fixture(scope="module")
def jb():
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def test_calls_of_more_work_items_than_a_launch_has(jb):
    """A launch has fewer than 2^32 work-items, 2^24 workgroups of 256: what needs more is refused
    by the library, with its own message, before anything is launched."""
    def size(f32, total, packed, **kw):
        s = jb.AttnShape(65535, 1, 256, 256, 64, 0, 16, 8, 20, 0, 0, f32, f32, 0, 0, 0, 0, 0)
        for k, v in kw.items():
            setattr(s, k, v)
        n = ctypes.c_size_t(0)
        return jb.library().jb_attn_paged_workspace_size(ctypes.byref(s), total, packed, ctypes.byref(n))
    # fp32: a tile of 16 query rows for each sequence, and one for 16 tokens in a packed batch, times 256 heads
    assert size(jb.JB_F32, 15, 1) == 0                       # 65535 x 256 = 2^24 - 256
    assert size(jb.JB_F32, 16, 1) == 2                       # 2^24
    assert "more workgroups than a launch" in jb.last_error()
    assert size(jb.JB_F32, 131070, 1, T=2) == 2
    assert size(jb.JB_F32, 65535, 0) == 0
    assert size(jb.JB_BF16, 65535, 0) == 0                   # decode, a workgroup for each sequence and head
    assert size(jb.JB_BF16, 65535 * 40, 0, T=40) == 0
    assert size(jb.JB_BF16, 65535 * 140, 0, T=140) == 2      # two tiles each
    good = ctypes.c_void_p(0x10000)
    s = jb.AttnShape(1, (1 << 27) - 7, 1, 1, 256, 64, 0, 0, 0, 0, 0, jb.JB_BF16, jb.JB_BF16, 0, 0, 0, 0, 0)
    rope = jb.library().jb_qk_norm_rope
    assert rope(ctypes.byref(s), good, good, good, good, good, good, 1e-6, good, good, None) == 2   # 8 tokens a workgroup
    assert "more workgroups than a launch" in jb.last_error()


def test_a_stride_of_one_head_or_page_says_nothing(jb):
    """Tensors whose strides differ from the usual ones only where a dimension has one entry."""
    bf = torch.bfloat16
    x = torch.zeros(1, 6, 64, dtype=bf).transpose(0, 1)                 # [6, 1, 64], heads 384 apart
    assert x.stride(1) != 64 and x.is_contiguous() and jb._rows(x, "k")[1:] == (6, 64)
    wide = torch.zeros(6, 256, dtype=bf)[:, None, 64:128]               # a slice of one projection's output
    assert wide.stride(1) != 64 and jb._rows(wide, "k")[1:] == (6, 256)
    assert jb._rows(wide.unsqueeze(0), "k")[1:] == (6, 256)
    assert jb._rows(torch.zeros(3, 2, 256, dtype=bf)[:, :, None, :64], "k")[1:] == (6, 256)
    with pytest.raises(ValueError):
        jb._rows(torch.zeros(6, 2, 128, dtype=bf)[..., :64], "k")      # two heads that are not next to each other
    table, kv = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(1, 2, 16, 64, dtype=bf)
    v = torch.zeros(1, 4, 16, 64, dtype=bf)[:, :2]                      # one page: the distance to the next is nobody's
    assert k.stride() != v.stride() and jb._pages(k, v, table, kv, 3, 64) == (1, 2, 16, 0, 4)
    k = torch.zeros(5, 1, 16, 64, dtype=bf)
    v = torch.zeros(1, 5, 16, 64, dtype=bf).transpose(0, 1)
    assert k.stride() != v.stride() and jb._pages(k, v, table, kv, 3, 64) == (5, 1, 16, 1024, 4)
    with pytest.raises(ValueError):
        jb._pages(k, torch.zeros(5, 2, 16, 64, dtype=bf)[:, :1], table, kv, 3, 64)


class _Stream:
    """What the binding looks at of a torch stream, and the context torch would enter for it."""

    def __init__(self, device):
        self.device, self.cuda_stream = torch.device(device), 7


def test_stream_of_another_device_is_refused(jb, monkeypatch):
    """A call runs on q's device: a stream of another one cannot order it, and is not passed over."""
    import contextlib
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s) or contextlib.nullcontext())

    class Q:
        is_cuda, device = True, torch.device("cuda:1")
        get_device = staticmethod(lambda: 1)
    ran = lambda **kw: kw
    mine = _Stream("cuda:1")
    assert jb._on_stream(ran, dict(q=Q, stream=mine, k=3)) == dict(q=Q, k=3) and entered == [mine]
    with pytest.raises(ValueError, match="stream"):
        jb._on_stream(ran, dict(q=Q, stream=_Stream("cuda:0")))
    assert entered == [mine]
    with pytest.raises(ValueError, match="device tensors"):
        jb._on_stream(ran, dict(q=torch.zeros(1), stream=_Stream("cuda:0")))


def test_packed_rows_behind_the_last_sequence_need_no_longer_hint(jb):
    """A packed batch may have rows that no sequence owns, more of them than B max_seqlen leaves room
    for: the planned length grows, so that the library takes the call."""
    def plan(n, B, most):
        return jb._batch(torch.zeros(n, 2, 64), torch.zeros(B + 1, dtype=torch.int32), most)
    assert plan(100, 4, 60) == (4, 60) and plan(100, 4, None) == (4, 100) and plan(100, 4, 1000) == (4, 100)
    assert plan(8, 4, 2) == (4, 2)
    for n, B, most in ((9, 4, 2), (8, 3, 1), (64, 4, 1), (5, 4, 0)):
        b, t = plan(n, B, most)
        assert b == B and t == -(-n // B)
        s = jb.AttnShape(B, t, 2, 2, 64, 0, 16, 8, 20, 0, 0, jb.JB_BF16, jb.JB_BF16, 0, 0, 0, 0, 0)
        jb.attn_paged_workspace_size(s, n, True)   # (raises for a total that the shape cannot hold)
    assert plan(0, 4, 7) == (4, 0)
    with pytest.raises(ValueError, match="max_seqlen"):
        plan(8, 4, -1)
