"""CPU checks of the entry points for long contexts (a cache in 8 bits, selected pages): every bad
argument comes back as a status with a message that names it, before the HIP runtime is reached,
and the binding refuses tensors that do not fit.  Also the oracle's codes against torch's."""
import ctypes
import inspect

import numpy as np
import pytest
import torch

from oracle import blocks as ref8

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
GOOD = 0x10000
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def jb():
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def shape(jb, name="", **kw):
    s = jb.AttnShape(2, 5, 4, 2, 64, 64, 16, 8, 20, 0, 0, jb.JB_BF16, jb.JB_BF16, 0, 0, 0, 0, 0)
    if name in ("jb_block_scores", "jb_attn_blocks"):
        s.flags = jb.CACHE_E4M3
    for k, v in kw.items():
        setattr(s, k, v)
    return s


# as in test_layer_abi: T the token count, a number a required pointer's alignment, a negative one an
# optional one's, f a float, L the distance of scales, c / r count and the like, w a workspace size
CALLS = {
    "jb_qk_norm_rope_paged8": ("T", -4, 4, 4, 16, 16, 16, -16, -16, 4, -4, "f", 16, 16, 16, 1, 1, "L", "s"),
    "jb_attn_paged8": ("T", -4, 4, 4, 16, 16, 16, 1, 1, "L", "f", 16, -4, -256, "w", "s"),
    "jb_block_scores": ("T", -4, 4, 4, 16, 16, 1, "L", 16, -4, "s"),
    "jb_block_select": ("T", -4, 4, 4, "c", "r0", "r1", 4, "s"),
    "jb_attn_blocks": ("T", -4, 4, 4, 16, 16, 16, 1, 1, "L", 4, "c", "f", 16, -4, 256, "w", "s"),
}
CACHED = [n for n in CALLS if n != "jb_block_select"]


def call(jb, name, s, total=10, f=1e-6, ws=1 << 40, at=None, value=GOOD, L=0, count=None, first=1, recent=1):
    args = []
    if count is None:  # (lists of more than 2048 entries need a workspace)
        count = 3000 if name == "jb_attn_blocks" else 3
    for i, k in enumerate(CALLS[name]):
        args.append({"T": lambda: ctypes.c_int64(total), "f": lambda: ctypes.c_float(f), "w": lambda: ctypes.c_size_t(ws),
                     "s": lambda: P(None), "L": lambda: ctypes.c_int64(L), "c": lambda: ctypes.c_int32(count),
                     "r0": lambda: ctypes.c_int32(first), "r1": lambda: ctypes.c_int32(recent)}
                    .get(k, lambda: P(value if i == at else GOOD))())
    return getattr(jb.library(), name)(None if s is None else ctypes.byref(s), *args)


@pytest.mark.parametrize("name", list(CALLS))
def test_pointers(jb, name):
    s = shape(jb, name)
    for i, k in enumerate(CALLS[name]):
        if not isinstance(k, int):
            continue
        align = abs(k)
        if align > 1:
            assert call(jb, name, s, at=i, value=GOOD + align // 2) == INVALID, (i, jb.last_error())
            assert f"{align}-byte aligned" in jb.last_error() and name in jb.last_error()
        if k == 256:
            assert call(jb, name, s, at=i, value=None) == WORKSPACE, jb.last_error()
        elif k > 0:
            assert call(jb, name, s, at=i, value=None) == INVALID, (i, jb.last_error())
            assert "is NULL" in jb.last_error()
    assert call(jb, name, None) == INVALID and "shape is NULL" in jb.last_error()


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("field,value,status", [
    ("B", 0, INVALID), ("B", 65536, UNSUPPORTED), ("T", -1, INVALID), ("T", (1 << 30) + 1, UNSUPPORTED),
    ("H", 0, UNSUPPORTED), ("H", 257, UNSUPPORTED), ("Hkv", 3, UNSUPPORTED), ("Hkv", 0, UNSUPPORTED),
    ("D", 96, UNSUPPORTED), ("io_dtype", 2, INVALID), ("out_dtype", -1, INVALID), ("q_stride", 4 * 64 - 8, INVALID),
    ("q_stride", 4 * 64 + 4, INVALID), ("q_stride", 1 << 40, UNSUPPORTED),
    ("page", 8, UNSUPPORTED), ("page", 48, UNSUPPORTED), ("page", 8192, UNSUPPORTED),
    ("max_pages", 0, INVALID), ("max_pages", (1 << 26) + 1, UNSUPPORTED), ("num_pages", 0, INVALID),
    ("page_stride", 2 * 16 * 64 - 16, INVALID), ("page_stride", 2 * 16 * 64 + 2, INVALID), ("page_stride", 1 << 40, UNSUPPORTED),
    ("window", -1, INVALID), ("max_kv", -1, INVALID), ("flags", 64, INVALID),
])
def test_shape(jb, name, field, value, status):
    s = shape(jb, name, **{field: value})
    assert call(jb, name, s, total=s.B * s.T) == status, jb.last_error()
    assert field in jb.last_error() or "sizes exceed" in jb.last_error()


def test_bytes_of_a_cache_in_8_bits(jb):
    """A page's distance counts bytes: 16 of them, where 8 elements of bf16 are as many."""
    for name in CACHED:
        assert call(jb, name, shape(jb, name, page_stride=2 * 16 * 64 + 8)) == INVALID and "page_stride" in jb.last_error()
        for stride, status in ((1, INVALID), (-2, INVALID), (1 << 40, UNSUPPORTED)):
            assert call(jb, name, shape(jb, name), L=stride) == status, (name, stride)
            assert "scale_stride" in jb.last_error() or "sizes exceed" in jb.last_error()


@pytest.mark.parametrize("name", list(CALLS))
def test_tokens(jb, name):
    assert call(jb, name, shape(jb, name), total=11) == INVALID and "total_tokens" in jb.last_error()
    assert call(jb, name, shape(jb, name), total=-1) == INVALID
    assert call(jb, name, shape(jb, name), total=9, at=1, value=None) == INVALID   # dense: all of B T
    assert call(jb, name, shape(jb, name), total=0) == OK
    assert call(jb, name, shape(jb, name, B=65535, T=1 << 20), total=1 << 31) == UNSUPPORTED


def test_append_arguments(jb):
    name = "jb_qk_norm_rope_paged8"
    for rot in (8, 72, 80, -16):
        assert call(jb, name, shape(jb, rot=rot)) == UNSUPPORTED and "rot" in jb.last_error()
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(jb, name, shape(jb), f=eps) == INVALID and "eps" in jb.last_error()
    assert call(jb, name, shape(jb, flags=jb.ROPE_NO_NORM)) == INVALID and "must be NULL" in jb.last_error()
    assert call(jb, name, shape(jb, out_dtype=jb.JB_F32)) == UNSUPPORTED and "out_dtype" in jb.last_error()
    # 16 rows a workgroup and key head
    s = shape(jb, B=1, T=1 << 20, H=256, Hkv=256, D=64)
    assert call(jb, name, s, total=1 << 20) == UNSUPPORTED and "more workgroups" in jb.last_error()


def test_attention_arguments(jb):
    for name in ("jb_attn_paged8", "jb_attn_blocks"):
        for scale in (-0.5, float("nan"), float("inf")):
            assert call(jb, name, shape(jb, name), f=scale) == INVALID and "scale" in jb.last_error()
    n = ctypes.c_size_t(7)
    s = shape(jb, max_pages=4096)
    size = jb.library().jb_attn_paged8_workspace_size
    assert size(ctypes.byref(s), 10, 0, ctypes.byref(n)) == OK and n.value > 0
    assert call(jb, "jb_attn_paged8", s, at=1, value=None, ws=n.value - 1) == WORKSPACE and str(n.value) in jb.last_error()
    assert size(ctypes.byref(s), 10, 0, None) == INVALID
    assert size(ctypes.byref(s), 0, 1, ctypes.byref(n)) == OK and n.value == 0
    size = jb.library().jb_attn_blocks_workspace_size
    for flags in (0, jb.CACHE_E4M3):
        s = shape(jb, flags=flags)
        assert size(ctypes.byref(s), 10, 0, 3, ctypes.byref(n)) == OK and n.value == 0      # one piece of a short list
        assert size(ctypes.byref(shape(jb, flags=flags, B=1, T=1, max_pages=400)), 1, 0, 300, ctypes.byref(n)) == OK
        assert n.value >= 2 * 4 * (64 + 2) * 4                                              # pieces of a long one
        assert size(ctypes.byref(s), 10, 0, 3000, ctypes.byref(n)) == OK and n.value >= 10 * 2 * 3001 * 4
    assert call(jb, "jb_attn_blocks", s, ws=n.value - 1) == WORKSPACE and str(n.value) in jb.last_error()
    assert size(ctypes.byref(s), 10, 0, 3, None) == INVALID
    assert size(ctypes.byref(s), 0, 1, 3, ctypes.byref(n)) == OK and n.value == 0


def test_max_kv_is_no_part_of_lists(jb):
    """The workspace of jb_attn_blocks (short lists, long ones, fp32) does not depend on max_kv."""
    size, n = jb.library().jb_attn_blocks_workspace_size, ctypes.c_size_t(0)
    for io, count in ((jb.JB_BF16, 300), (jb.JB_BF16, 3000), (jb.JB_F32, 300), (jb.JB_F32, 3000)):
        got = set()
        for max_kv in (0, 1, 1 << 20):
            s = shape(jb, B=1, T=1, page=64, max_pages=4096, num_pages=4096, io_dtype=io, max_kv=max_kv)
            assert size(ctypes.byref(s), 1, 0, count, ctypes.byref(n)) == OK
            got.add(n.value)
        assert len(got) == 1, (io, count, got)


def test_block_arguments(jb):
    for name in ("jb_block_scores", "jb_attn_blocks"):
        assert call(jb, name, shape(jb, flags=0)) == INVALID and "must be NULL" in jb.last_error()
        assert call(jb, name, shape(jb, name, window=5)) == UNSUPPORTED and "window" in jb.last_error()
    assert call(jb, "jb_block_select", shape(jb, window=5)) == UNSUPPORTED
    assert call(jb, "jb_block_select", shape(jb, flags=jb.CACHE_E4M3)) == INVALID
    for count, first, recent in ((0, 0, 1), (-1, 0, 1), (3, -1, 1), (3, 0, 0), (3, 2, 2), (3, 0x7fffffff, 0x7fffffff)):
        assert call(jb, "jb_block_select", shape(jb), count=count, first=first, recent=recent) == INVALID
    assert call(jb, "jb_block_select", shape(jb, max_pages=65537)) == UNSUPPORTED and "65536" in jb.last_error()
    assert call(jb, "jb_attn_blocks", shape(jb, "jb_attn_blocks"), count=0) == INVALID and "count" in jb.last_error()
    assert call(jb, "jb_attn_blocks", shape(jb, "jb_attn_blocks"), count=(1 << 26) + 1) == UNSUPPORTED
    s = shape(jb, "jb_block_scores", B=1, T=1 << 20, H=256, Hkv=256)
    for name in ("jb_block_scores", "jb_block_select", "jb_attn_blocks"):
        s.flags = shape(jb, name).flags
        assert call(jb, name, s, total=1 << 20) == UNSUPPORTED and "more workgroups" in jb.last_error()
    # 1024 threads a row from 4097 pages on
    s = shape(jb, B=1, T=1 << 22, H=1, Hkv=1, max_pages=4097)
    assert call(jb, "jb_block_select", s, total=1 << 22) == UNSUPPORTED and "more workgroups" in jb.last_error()

    # one token of 65535 packed sequences, fp32: a sequence has a place of its own even without tokens
    s = shape(jb, "jb_block_scores", B=65535, T=1, H=1, Hkv=1, max_pages=65536, io_dtype=jb.JB_F32)
    assert call(jb, "jb_block_scores", s, total=1) == UNSUPPORTED and "more workgroups" in jb.last_error()


def test_binding(jb):
    P_, Hkv, page, D = 5, 2, 32, 64
    k = torch.zeros(P_, Hkv, page // 16, dtype=torch.uint8).view(E8M0)
    assert jb._scales(k, k, "s", P_, Hkv, page) == Hkv * page // 16
    both = torch.zeros(P_, 3, Hkv, page // 16, dtype=torch.uint8).view(E8M0)
    assert jb._scales(both[:, 1], both[:, 2], "s", P_, Hkv, page) == 3 * Hkv * page // 16
    assert jb._scales(k[:1], None, "s", 1, Hkv, page) == 0
    for a, b in ((k[:4], k[:4]), (k, k[:4]), (both[:, 1], k), (both[:, :2, 0], None), (k[:1].expand(P_, Hkv, 2), None)):
        with pytest.raises(ValueError):
            jb._scales(a, b, "s", P_, Hkv, page)
    bf = torch.bfloat16
    c = torch.zeros(1)
    assert [g[0] for g in jb._cache_of(bf, c, None)] == [bf] and [g[0] for g in jb._cache_of(bf, c, k, c, k)] == [E4M3, E8M0]
    for ks, vs in ((k, None), (None, k)):
        with pytest.raises(ValueError, match="go together"):
            jb._cache_of(bf, c, ks, c, vs)
    with pytest.raises(ValueError, match="device tensors"):
        jb.block_select(torch.zeros(2, 1, 4), torch.zeros(2, dtype=torch.int32), 2, 16)


def test_numbers_past_32_bits(jb):
    """They are refused, not taken for what their low 32 bits are."""
    scores, kv, big = torch.zeros(2, 1, 4), torch.zeros(2, dtype=torch.int32), (1 << 32) + 16
    for count, page, first, recent, name in ((big, 16, 1, 1, "count"), (2, big, 1, 1, "page"), (2, 16, 1 << 32, 1, "first"),
                                             (2, 16, 0, (1 << 32) + 1, "recent"), (2, 16, -(1 << 32), 1, "first")):
        with pytest.raises(ValueError, match=name):
            jb.block_select(scores, kv, count, page, first=first, recent=recent)
    q, c = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(1, 1, 1, dtype=torch.int32).expand(2, 1, big)
    with pytest.raises(ValueError, match="count"):
        jb.attn_blocks(q, c, c, torch.zeros(2, 3, dtype=torch.int32), kv, blocks)


@pytest.mark.parametrize("name", ["qk_norm_rope_paged8", "attn_paged8", "block_scores", "block_select", "attn_blocks"])
def test_stream_argument_is_taken(jb, monkeypatch, name):
    fn, seen = getattr(jb, name), []
    monkeypatch.setattr(jb, "_on_stream", lambda f, args, *first: seen.append((f, dict(args))) or "there")
    given = {n: object() for n, p in inspect.signature(fn).parameters.items()}
    assert fn(**given) == "there" and seen == [(fn, given)]
    assert "return _on" not in fn.__doc__ and fn.__doc__.rstrip().endswith(".")


def test_codes_of_the_oracle():
    """The oracle's e4m3 against torch's type: every code, and roundings next to every border."""
    assert np.array_equal(ref8.E4M3, torch.arange(256, dtype=torch.uint8).view(E4M3).double().numpy(), equal_nan=True)
    v = ref8.E4M3[:127]
    mid = (v[:-1] + v[1:]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0, dtype=np.float32), np.nextafter(mid, 500, dtype=np.float32)])
    x = np.concatenate([x, -x]).astype(np.float32)
    assert np.array_equal(ref8.encode(x), torch.from_numpy(x).to(E4M3).view(torch.uint8).numpy())
    assert np.isnan(ref8.E4M3[ref8.encode([np.nan, np.inf, -np.inf])]).all()
    assert [ref8.exponent(m) for m in (0, 448, 448.01, 224, 224.01, 3.4e38, 1e-44)] == [1, 127, 128, 126, 127, 247, 1]
    e = torch.arange(1, 255, dtype=torch.uint8)
    assert np.array_equal(ref8.scale_value(e.numpy()), e.view(E8M0).double().numpy())
    x = np.array([1.0, 3, 3, -np.inf, np.nan, 2, 9, 0])
    assert ref8.select(x, 6, 4, 1, 2) == [0, 1, 5, 6] and ref8.select(x, 2, 4, 0, 1) == [0, 1, 2, -1]
    assert ref8.select(x, 7, 7, 0, 1) == [0, 1, 2, 3, 5, 6, 7] and ref8.counting([3, 3, 1, 9, 5, -1, 6], 6) == [3, 5, 6]
