"""CPU checks of the attention-layer entry points: every bad argument comes back as a status
with a message that names it, before the HIP runtime is reached, and the binding refuses
tensors that do not fit (this machine may have no GPU; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
GOOD = 0x10000


@pytest.fixture(scope="module")
def jb():
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


def shape(jb, **kw):
    s = jb.AttnShape(2, 5, 4, 2, 64, 64, 16, 8, 20, 0, 0, jb.JB_BF16, jb.JB_BF16, 0, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


# name: arguments after the shape: T the token count, 16 / 4 / 256 a required pointer's alignment,
# -16 / -4 an optional one, f a float, w a workspace size, s the stream
CALLS = {
    "jb_qk_norm_rope": (16, 16, -16, -16, 4, 4, "f", 16, 16, "s"),
    "jb_qk_norm_rope_backward": (16, 16, -16, -16, 4, 4, "f", 16, 16, 16, 16, -4, -4, 256, "w", "s"),
    "jb_qk_norm_rope_paged": ("T", -4, 4, 4, 16, 16, 16, -16, -16, 4, -4, "f", 16, 16, 16, "s"),
    "jb_attn_paged": ("T", -4, 4, 4, 16, 16, 16, "f", 16, -4, -256, "w", "s"),
}


def call(jb, name, s, total=10, f=1e-6, ws=1 << 40, at=None, value=GOOD):
    args = []
    for i, k in enumerate(CALLS[name]):
        args.append(ctypes.c_int64(total) if k == "T" else ctypes.c_float(f) if k == "f" else
                    ctypes.c_size_t(ws) if k == "w" else P(None) if k == "s" else P(value if i == at else GOOD))
    return getattr(jb.library(), name)(None if s is None else ctypes.byref(s), *args)


@pytest.mark.parametrize("name", list(CALLS))
def test_pointers(jb, name):
    s = shape(jb)
    for i, k in enumerate(CALLS[name]):
        if not isinstance(k, int):
            continue
        align = abs(k)
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
    ("Hkv", -2, UNSUPPORTED), ("D", 96, UNSUPPORTED), ("D", 0, UNSUPPORTED), ("io_dtype", 2, INVALID),
    ("out_dtype", -1, INVALID), ("q_stride", 4 * 64 - 8, INVALID), ("q_stride", 4 * 64 + 4, INVALID),
    ("q_stride", -256, INVALID), ("k_stride", 64, INVALID), ("v_stride", 130, INVALID), ("q_stride", 1 << 40, UNSUPPORTED),
])
def test_shape(jb, name, field, value, status):
    s = shape(jb, **{field: value})
    assert call(jb, name, s, total=s.B * s.T) == status, jb.last_error()
    text = jb.last_error()
    assert field in text or "sizes exceed" in text, text


@pytest.mark.parametrize("name", ["jb_qk_norm_rope", "jb_qk_norm_rope_backward", "jb_qk_norm_rope_paged"])
def test_rotation(jb, name):
    for rot in (8, 72, 80, -16):
        assert call(jb, name, shape(jb, rot=rot)) == UNSUPPORTED and "rot" in jb.last_error()
    assert call(jb, name, shape(jb, flags=4)) == INVALID and "flags" in jb.last_error()
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(jb, name, shape(jb), f=eps) == INVALID and "eps" in jb.last_error()
    assert call(jb, name, shape(jb, flags=jb.ROPE_NO_NORM)) == INVALID and "must be NULL" in jb.last_error()


@pytest.mark.parametrize("name", ["jb_qk_norm_rope_paged", "jb_attn_paged"])
@pytest.mark.parametrize("field,value,status", [
    ("page", 8, UNSUPPORTED), ("page", 48, UNSUPPORTED), ("page", 8192, UNSUPPORTED), ("page", 0, UNSUPPORTED),
    ("max_pages", 0, INVALID), ("max_pages", (1 << 26) + 1, UNSUPPORTED), ("num_pages", 0, INVALID),
    ("page_stride", 2 * 16 * 64 - 8, INVALID), ("page_stride", 2 * 16 * 64 + 2, INVALID), ("page_stride", 1 << 40, UNSUPPORTED),
    ("num_pages", 1 << 30, UNSUPPORTED), ("window", -1, INVALID), ("max_kv", -1, INVALID),
])
def test_cache(jb, name, field, value, status):
    assert call(jb, name, shape(jb, **{field: value})) == status, jb.last_error()


def test_tokens(jb):
    for name in ("jb_qk_norm_rope_paged", "jb_attn_paged"):
        assert call(jb, name, shape(jb), total=11) == INVALID and "total_tokens" in jb.last_error()
        assert call(jb, name, shape(jb), total=-1) == INVALID
        # dense: all of B T
        assert call(jb, name, shape(jb), total=9, at=1, value=None) == INVALID
        assert call(jb, name, shape(jb), total=0) == OK     # nothing to do
        assert call(jb, name, shape(jb, B=65535, T=1 << 20), total=1 << 31) == UNSUPPORTED
    assert call(jb, "jb_qk_norm_rope", shape(jb, T=0)) == OK


def test_attention_arguments(jb):
    for scale in (-0.5, float("nan"), float("inf")):
        assert call(jb, "jb_attn_paged", shape(jb), f=scale) == INVALID and "scale" in jb.last_error()
    assert call(jb, "jb_attn_paged", shape(jb, flags=1)) == INVALID
    n = ctypes.c_size_t(7)
    size = jb.library().jb_attn_paged_workspace_size
    one = shape(jb, max_pages=1)
    assert size(ctypes.byref(one), 10, 0, ctypes.byref(n)) == OK and n.value == 0      # one piece
    s = shape(jb, max_pages=4096)
    assert size(ctypes.byref(s), 10, 0, ctypes.byref(n)) == OK and n.value >= 2 * 10 * 4 * 64 * 4
    assert call(jb, "jb_attn_paged", s, at=1, value=None, ws=n.value - 1) == WORKSPACE
    assert str(n.value) in jb.last_error()
    assert size(ctypes.byref(s), 10, 0, None) == INVALID
    assert size(ctypes.byref(s), 0, 1, ctypes.byref(n)) == OK and n.value == 0


def test_backward_workspace(jb):
    n = ctypes.c_size_t(0)
    s = shape(jb, T=1000)
    assert jb.library().jb_qk_norm_rope_backward_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0
    assert call(jb, "jb_qk_norm_rope_backward", s, ws=n.value - 1) == WORKSPACE and str(n.value) in jb.last_error()
    # more workgroups than a launch takes are not asked for: the pass strides over its tokens
    s = shape(jb, B=1, T=1 << 30, H=1, Hkv=1)
    assert jb.library().jb_qk_norm_rope_backward_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK
    assert n.value <= 1 << 20


def test_binding_refuses_what_does_not_fit(jb):
    bf = torch.bfloat16
    q, k = torch.zeros(6, 4, 64, dtype=bf), torch.zeros(6, 2, 64, dtype=bf)
    pos, fr = torch.zeros(6, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="device tensors"):
        jb.qk_norm_rope(q, k, pos, fr)
    # shape and dtype checks, on the meta device's stand-in for one
    rows = jb._rows
    assert rows(q, "q")[1:] == (6, 256) and rows(q[:1], "q")[1:] == (1, 0)
    assert rows(q.view(2, 3, 4, 64), "q")[1:] == (6, 256)
    wide = torch.zeros(6, 8, 64, dtype=bf)
    assert rows(wide[:, :4], "q")[1:] == (6, 512) and rows(wide.view(2, 3, 8, 64)[:, :, 2:4], "q")[1:] == (6, 512)
    for bad in (q[..., ::2], q.transpose(1, 2), q[:1].expand(6, 4, 64), q[0], wide.view(3, 2, 8, 64)[:, :1].expand(3, 2, 8, 64),
                torch.zeros(4, 6, 4, 64)[:, ::4]):
        with pytest.raises(ValueError):
            rows(bad, "q")
    kc = torch.zeros(5, 2, 16, 64, dtype=bf)
    table, kv = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    assert jb._pages(kc, kc, table, kv, 3, 64) == (5, 2, 16, 2048, 4)
    layers = torch.zeros(5, 3, 2, 16, 64, dtype=bf)
    assert jb._pages(layers[:, 1], layers[:, 2], table, kv, 3, 64)[3] == 3 * 2048
    for args in ((kc, kc[:4], table, kv, 3, 64), (kc, kc, table, kv, 2, 64), (kc, kc, table, kv[:2], 3, 64),
                 (kc, kc, table, kv, 3, 128), (kc.transpose(1, 2), kc.transpose(1, 2), table, kv, 3, 64),
                 (kc[:1].expand(5, 2, 16, 64), kc[:1].expand(5, 2, 16, 64), table, kv, 3, 64)):
        with pytest.raises(ValueError):
            jb._pages(*args)
    jb._same(-1, (bf, "k v", (k, None)), (torch.int32, "kv_lens", (kv,)))
    with pytest.raises(TypeError, match="kv_lens: expected torch.int32"):
        jb._same(-1, (bf, "k v", (k, None)), (torch.int32, "table kv_lens", (table, kv.long())))
    with pytest.raises(ValueError, match="v is on cpu"):
        jb._same(0, (bf, "k v", (None, k)))
    with pytest.raises(TypeError):
        jb._code(torch.float16)
    with pytest.raises(ValueError):
        jb._flat(q[:, :2], "q", 6, 2, 64)


@pytest.mark.parametrize("name", ["qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_paged", "attn_paged"])
def test_stream_argument_is_taken(jb, monkeypatch, name):
    """With a stream every call goes through the stream's own context, its other arguments as given;
    the documentation holds nothing but words."""
    import inspect
    fn, seen = getattr(jb, name), []
    monkeypatch.setattr(jb, "_on_stream", lambda f, args: seen.append((f, dict(args))) or "there")
    given = {n: object() for n, p in inspect.signature(fn).parameters.items()}
    assert fn(**given) == "there" and seen == [(fn, given)]
    assert "return _on" not in fn.__doc__ and fn.__doc__.rstrip().endswith(".")
