"""ctypes binding of libjetblock (include/jetblock.h).

Argument marshalling only: shapes and dtypes are read off torch tensors,
outputs and workspaces are allocated with torch on the tensors' device, and
every computation runs in the library's HIP kernels on the current torch
stream.  There is no fallback: if libjetblock.so is missing or fails to load,
importing this module raises, and a call on CPU tensors raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libjetblock.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "jetblock.h")

JB_OK, JB_ERR_INVALID_ARG, JB_ERR_UNSUPPORTED, JB_ERR_WORKSPACE, JB_ERR_HIP = range(5)
JB_BF16, JB_F32 = 0, 1
_DT = {torch.bfloat16: JB_BF16, torch.float32: JB_F32}
_TORCH = {JB_BF16: torch.bfloat16, JB_F32: torch.float32}


class JetBlockError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{status}]")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H", "dk", "dv", "d_model", "gen_hidden", "taps", "chunk",
                 "io_dtype", "out_dtype", "flags")]


class AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H", "Hkv", "D", "rot", "page", "max_pages", "num_pages", "max_kv", "window",
                 "io_dtype", "out_dtype", "flags")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "page_stride")]


ROPE_INTERLEAVED, ROPE_NO_NORM = 1, 2


def flag_segment(n: int) -> int:
    return (int(n) & 0xFFFF) << 8


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libjetblock.so not built at {LIB_PATH}; run "
                      "`python -m gated_delta_rule_jetblock_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_S = ctypes.POINTER(Shape)
_SZ = ctypes.c_size_t
_lib.jb_status_string.argtypes = [ctypes.c_int]
_lib.jb_status_string.restype = ctypes.c_char_p
_lib.jb_last_error.argtypes = []
_lib.jb_last_error.restype = ctypes.c_char_p
_lib.jb_version.argtypes = []
_lib.jb_version.restype = ctypes.c_int32
_lib.jb_prefill_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_decode_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_prefill.argtypes = [_S] + [_P] * 15 + [_P, _SZ, _P]
_lib.jb_decode_step.argtypes = [_S] + [_P] * 15 + [_P, _SZ, _P]
_lib.jb_prefill_noalloc.argtypes = [_S] + [_P] * 15 + [_P]
_lib.jb_gen_taps.argtypes = [_S] + [_P] * 6 + [_P]
_lib.jb_gen_conv.argtypes = [_S] + [_P] * 9 + [_P]
_lib.jb_prologue.argtypes = [_S] + [_P] * 6 + [_P]
_lib.jb_probe_mfma.argtypes = [ctypes.c_int32, _P, _P, _P, _P]
_lib.jb_decode_update.argtypes = [_S] + [_P] * 11 + [_P]
_lib.jb_project_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_prefill_from_x_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_project.argtypes = [_S] + [_P] * 18 + [_P, _SZ, _P]
_lib.jb_prefill_from_x.argtypes = [_S] + [_P] * 17 + [_P, _SZ, _P]
_lib.jb_decode_step_from_x_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_decode_step_from_x.argtypes = [_S] + [_P] * 17 + [_P, _SZ, _P]
_lib.jb_prefill_static_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_prefill_static.argtypes = [_S] + [_P] * 17 + [_P, _SZ, _P]
_lib.jb_decode_step_static.argtypes = [_S] + [_P] * 17 + [_P]
_lib.jb_prefill_varlen_workspace_size.argtypes = [_S, ctypes.c_int64, ctypes.POINTER(_SZ)]
_lib.jb_prefill_varlen.argtypes = [_S, ctypes.c_int64] + [_P] * 16 + [_P, _SZ, _P]
_lib.jb_backward_workspace_size.argtypes = [_S, ctypes.POINTER(_SZ)]
_lib.jb_backward.argtypes = [_S] + [_P] * 27 + [_P, _SZ, _P]
_A = ctypes.POINTER(AttnShape)
_L, _F = ctypes.c_int64, ctypes.c_float
_lib.jb_qk_norm_rope.argtypes = [_A] + [_P] * 6 + [_F] + [_P] * 3
_lib.jb_qk_norm_rope_backward_workspace_size.argtypes = [_A, ctypes.POINTER(_SZ)]
_lib.jb_qk_norm_rope_backward.argtypes = [_A] + [_P] * 6 + [_F] + [_P] * 7 + [_SZ, _P]
_lib.jb_qk_norm_rope_paged.argtypes = [_A, _L] + [_P] * 10 + [_F] + [_P] * 4
_lib.jb_attn_paged_workspace_size.argtypes = [_A, _L, ctypes.c_int32, ctypes.POINTER(_SZ)]
_lib.jb_attn_paged.argtypes = [_A, _L] + [_P] * 6 + [_F] + [_P] * 3 + [_SZ, _P]
for _f in ("jb_qk_norm_rope", "jb_qk_norm_rope_backward_workspace_size", "jb_qk_norm_rope_backward",
           "jb_qk_norm_rope_paged", "jb_attn_paged_workspace_size", "jb_attn_paged",
           "jb_prefill_workspace_size", "jb_decode_workspace_size", "jb_prefill", "jb_prefill_noalloc",
           "jb_decode_step",
           "jb_gen_taps", "jb_gen_conv", "jb_prologue", "jb_probe_mfma", "jb_decode_update",
           "jb_project_workspace_size", "jb_prefill_from_x_workspace_size", "jb_project", "jb_prefill_from_x",
           "jb_decode_step_from_x_workspace_size", "jb_decode_step_from_x", "jb_prefill_static_workspace_size",
           "jb_prefill_static", "jb_decode_step_static", "jb_prefill_varlen_workspace_size",
           "jb_prefill_varlen", "jb_backward_workspace_size", "jb_backward"):
    getattr(_lib, _f).restype = ctypes.c_int


def declared_functions() -> list[str]:
    """Names of the functions include/jetblock.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(jb_[a-z_0-9]+)\s*\(", text)) - {"jb_FLAG_SEGMENT"})


def library() -> ctypes.CDLL:
    return _lib


def version() -> int:
    return _lib.jb_version()


def last_error() -> str:
    return _lib.jb_last_error().decode()


def _check(status: int):
    if status != JB_OK:
        raise JetBlockError(status, f"{_lib.jb_status_string(status).decode()}: {last_error()}")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError("libjetblock takes device tensors; got a tensor on " + str(t.device))
    if not t.is_contiguous():
        raise ValueError("libjetblock takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_shape(B, T, H, dk, dv, d_model, io_dtype=JB_BF16, out_dtype=JB_F32, flags=0) -> Shape:
    return Shape(B, T, H, dk, dv, d_model, 32, 4, 64, io_dtype, out_dtype, flags)


def _io_code(t: torch.Tensor) -> int:
    return _code(t.dtype)


def _code(dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def prefill_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_prefill_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def decode_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_decode_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device byte buffer of at least nbytes (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def prefill(x, q, k, v, alpha, beta, W1, W2, b1=None, b2=None, S0=None, conv_in=None, *,
            out_dtype=torch.float32, seg_len: int | None = None, o=None, S_final=None,
            conv_out=None, want_conv_out=True, ws=None, stream=None):
    """jb_prefill.  x [B,T,D], q,k [B,T,H,dk], v [B,T,H,dv], alpha,beta [B,T,H] f32.

    Returns dict(o, S_final, conv_out).  Outputs are allocated unless given.
    """
    B, T, D = x.shape
    H, dk = q.shape[2], q.shape[3]
    dv = v.shape[3]
    io = _io_code(x)
    shape = make_shape(B, T, H, dk, dv, D, io, _DT[out_dtype], flag_segment(seg_len) if seg_len else 0)
    dev = x.device
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    if S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if conv_out is None and want_conv_out:
        conv_out = torch.empty((B, 3, H, dv), dtype=x.dtype, device=dev)
    need = prefill_workspace_size(shape)
    if ws is None:
        ws = workspace(need, dev)
    _check(_lib.jb_prefill(ctypes.byref(shape), _ptr(x), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                           _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(S0), _ptr(conv_in), _ptr(o),
                           _ptr(S_final), _ptr(conv_out), _ptr(ws), ws.numel(), _stream(stream)))
    return dict(o=o, S_final=S_final, conv_out=conv_out)


def prefill_noalloc(x, q, k, v, alpha, beta, W1, W2, b1=None, b2=None, S0=None, conv_in=None, *,
                    out_dtype=torch.float32, seg_len: int | None = None, o=None, S_final=None,
                    conv_out=None, want_conv_out=True, stream=None):
    """jb_prefill_noalloc: jb_prefill on the library's own per-device scratch array
    (NOALLOC_SCRATCH_BYTES).  Same arguments as prefill() without ws; outputs are
    allocated here unless given, so a caller that must not allocate passes o, S_final
    and conv_out (or want_conv_out=False)."""
    B, T, D = x.shape
    H, dk = q.shape[2], q.shape[3]
    dv = v.shape[3]
    shape = make_shape(B, T, H, dk, dv, D, _io_code(x), _DT[out_dtype], flag_segment(seg_len) if seg_len else 0)
    dev = x.device
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    if S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if conv_out is None and want_conv_out:
        conv_out = torch.empty((B, 3, H, dv), dtype=x.dtype, device=dev)
    _check(_lib.jb_prefill_noalloc(ctypes.byref(shape), _ptr(x), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                   _ptr(beta), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(S0), _ptr(conv_in),
                                   _ptr(o), _ptr(S_final), _ptr(conv_out), _stream(stream)))
    return dict(o=o, S_final=S_final, conv_out=conv_out)


NOALLOC_SCRATCH_BYTES = 64 << 20


def decode_step(S, cache, x_t, q_t, k_t, v_t, alpha_t, beta_t, W1, W2, b1=None, b2=None, *,
                out_dtype=torch.float32, S_out=None, cache_out=None, o=None, ws=None, stream=None):
    """jb_decode_step.  S [B,H,dk,dv] f32, cache [B,3,H,dv], x_t [B,D], q_t,k_t [B,H,dk],
    v_t [B,H,dv], alpha_t,beta_t [B,H].  In place on S and cache unless S_out/cache_out
    are given.  Returns dict(o, S, cache)."""
    B, D = x_t.shape
    H, dk = q_t.shape[1], q_t.shape[2]
    dv = v_t.shape[2]
    shape = make_shape(B, 1, H, dk, dv, D, _io_code(x_t), _DT[out_dtype])
    if S_out is None:
        S_out = S
    if cache_out is None:
        cache_out = cache
    if o is None:
        o = torch.empty((B, H, dv), dtype=out_dtype, device=x_t.device)
    if ws is None and decode_workspace_size(shape) > 0:
        ws = workspace(decode_workspace_size(shape), x_t.device)
    _check(_lib.jb_decode_step(ctypes.byref(shape), _ptr(S), _ptr(S_out), _ptr(cache), _ptr(cache_out),
                               _ptr(x_t), _ptr(q_t), _ptr(k_t), _ptr(v_t), _ptr(alpha_t), _ptr(beta_t),
                               _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(o), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(stream)))
    return dict(o=o, S=S_out, cache=cache_out)


def decode_update(S, cache, q_t, k_t, v_t, alpha_t, beta_t, taps, *, d_model: int = 128,
                  out_dtype=torch.float32, S_out=None, cache_out=None, o=None, stream=None):
    """jb_decode_update: the state-update stage with taps [B,H,4] f32 precomputed.
    In place on S and cache unless S_out/cache_out are given."""
    B, H, dk = q_t.shape
    dv = v_t.shape[2]
    shape = make_shape(B, 1, H, dk, dv, d_model, _io_code(q_t), _DT[out_dtype])
    S_out = S if S_out is None else S_out
    cache_out = cache if cache_out is None else cache_out
    if o is None:
        o = torch.empty((B, H, dv), dtype=out_dtype, device=q_t.device)
    _check(_lib.jb_decode_update(ctypes.byref(shape), _ptr(S), _ptr(S_out), _ptr(cache), _ptr(cache_out),
                                 _ptr(q_t), _ptr(k_t), _ptr(v_t), _ptr(alpha_t), _ptr(beta_t), _ptr(taps),
                                 _ptr(o), _stream(stream)))
    return dict(o=o, S=S_out, cache=cache_out)


def gen_taps(x, W1, W2, b1=None, b2=None, H: int | None = None, *, out=None, stream=None):
    """jb_gen_taps on x [B,T,D] -> taps [B,T,H,4] f32 (written into `out` when given)."""
    B, T, D = x.shape
    if H is None:
        H = W2.shape[0] // 4
    shape = make_shape(B, T, H, 32, 64, D, _io_code(x))
    taps = torch.empty((B, T, H, 4), dtype=torch.float32, device=x.device) if out is None else out
    _check(_lib.jb_gen_taps(ctypes.byref(shape), _ptr(x), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(taps),
                            _stream(stream)))
    return taps


def gen_conv(x, W1, W2, v, b1=None, b2=None, conv_in=None, *, stream=None):
    """jb_gen_conv -> (taps [B,T,H,4], vconv [B,T,H,dv]) f32."""
    B, T, D = x.shape
    H, dv = v.shape[2], v.shape[3]
    shape = make_shape(B, T, H, 32, dv, D, _io_code(x))
    taps = torch.empty((B, T, H, 4), dtype=torch.float32, device=x.device)
    vconv = torch.empty((B, T, H, dv), dtype=torch.float32, device=x.device)
    _check(_lib.jb_gen_conv(ctypes.byref(shape), _ptr(x), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(v),
                            _ptr(conv_in), _ptr(taps), _ptr(vconv), _stream(stream)))
    return taps, vconv


def prologue(q, k, alpha, *, stream=None):
    """jb_prologue -> (qhat, khat [B,T,H,dk] f32, g [B,T,H] f32)."""
    B, T, H, dk = q.shape
    shape = make_shape(B, T, H, dk, 64, 128, _io_code(q))
    qh = torch.empty((B, T, H, dk), dtype=torch.float32, device=q.device)
    kh = torch.empty_like(qh)
    g = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    _check(_lib.jb_prologue(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(alpha), _ptr(qh), _ptr(kh), _ptr(g),
                            _stream(stream)))
    return qh, kh, g


def probe_mfma(kind: int, A, B, *, stream=None):
    """jb_probe_mfma: D = A B for A [16,32], B [32,16] f32 device tensors."""
    D = torch.empty((16, 16), dtype=torch.float32, device=A.device)
    _check(_lib.jb_probe_mfma(int(kind), _ptr(A), _ptr(B), _ptr(D), _stream(stream)))
    return D


def project_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_project_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def prefill_from_x_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_prefill_from_x_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def _proj_shape(x, Wq, Wv, Wa, seg_len=None, out_dtype=torch.float32):
    B, T, D = x.shape
    H = Wa.shape[0]
    dk = Wq.shape[0] // H
    dv = Wv.shape[0] // H
    return make_shape(B, T, H, dk, dv, D, JB_BF16, _DT[out_dtype],
                      flags=flag_segment(seg_len) if seg_len else 0)


def project(x, Wq, Wk, Wv, Wa, Wb, W1, W2, ba=None, bb=None, b1=None, b2=None, *, ws=None, stream=None):
    """jb_project.  x [B,T,D] bf16; Wq, Wk [H*dk,D], Wv [H*dv,D], Wa, Wb [H,D], W1 [32,D], W2 [4H,32]
    bf16.  Returns dict(q, k [B,T,H,dk], v [B,T,H,dv] bf16, alpha, beta [B,T,H], taps [B,T,H,4] f32)."""
    shape = _proj_shape(x, Wq, Wv, Wa)
    B, T, H, dk, dv = shape.B, shape.T, shape.H, shape.dk, shape.dv
    dev = x.device
    q = torch.empty((B, T, H, dk), dtype=torch.bfloat16, device=dev)
    k = torch.empty_like(q)
    v = torch.empty((B, T, H, dv), dtype=torch.bfloat16, device=dev)
    alpha = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    beta = torch.empty_like(alpha)
    taps = torch.empty((B, T, H, 4), dtype=torch.float32, device=dev)
    # the projection kernel takes no workspace (jb_project_workspace_size is 0)
    _check(_lib.jb_project(ctypes.byref(shape), _ptr(x), _ptr(Wq), _ptr(Wk), _ptr(Wv), _ptr(Wa), _ptr(ba),
                           _ptr(Wb), _ptr(bb), _ptr(W1), _ptr(b1), _ptr(W2),
                           _ptr(b2), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(taps), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream(stream)))
    return dict(q=q, k=k, v=v, alpha=alpha, beta=beta, taps=taps)


def prefill_from_x(x, Wq, Wk, Wv, Wa, Wb, W1, W2, ba=None, bb=None, b1=None, b2=None, S0=None, conv_in=None, *, out_dtype=torch.float32, seg_len: int | None = None,
                   o=None, S_final=None, conv_out=None, want_conv_out=True, ws=None, stream=None):
    """jb_prefill_from_x: the block from its layer input x (projections, generator, recurrence).
    Returns dict(o, S_final, conv_out)."""
    shape = _proj_shape(x, Wq, Wv, Wa, seg_len, out_dtype)
    B, T, H, dk, dv = shape.B, shape.T, shape.H, shape.dk, shape.dv
    dev = x.device
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    if S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if conv_out is None and want_conv_out:
        conv_out = torch.empty((B, 3, H, dv), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = workspace(prefill_from_x_workspace_size(shape), dev)
    _check(_lib.jb_prefill_from_x(ctypes.byref(shape), _ptr(x), _ptr(Wq), _ptr(Wk), _ptr(Wv), _ptr(Wa), _ptr(ba),
                                  _ptr(Wb), _ptr(bb), _ptr(W1), _ptr(b1), _ptr(W2),
                                  _ptr(b2), _ptr(S0), _ptr(conv_in), _ptr(o), _ptr(S_final), _ptr(conv_out),
                                  _ptr(ws), ws.numel(), _stream(stream)))
    return dict(o=o, S_final=S_final, conv_out=conv_out)


def decode_step_from_x_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_decode_step_from_x_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def decode_step_from_x(S, cache, x_t, Wq, Wk, Wv, Wa, Wb, W1, W2, ba=None, bb=None, b1=None, b2=None, *,
                       out_dtype=torch.float32, S_out=None, cache_out=None, o=None, ws=None, stream=None):
    """jb_decode_step_from_x: one decode step from the layer input x_t [B,D].  In place on S
    and cache unless S_out/cache_out are given.  Returns dict(o, S, cache)."""
    B, D = x_t.shape
    H = Wa.shape[0]
    dk, dv = Wq.shape[0] // H, Wv.shape[0] // H
    shape = make_shape(B, 1, H, dk, dv, D, JB_BF16, _DT[out_dtype])
    S_out = S if S_out is None else S_out
    cache_out = cache if cache_out is None else cache_out
    if o is None:
        o = torch.empty((B, H, dv), dtype=out_dtype, device=x_t.device)
    if ws is None:
        ws = workspace(decode_step_from_x_workspace_size(shape), x_t.device)
    _check(_lib.jb_decode_step_from_x(ctypes.byref(shape), _ptr(S), _ptr(S_out), _ptr(cache), _ptr(cache_out),
                                      _ptr(x_t), _ptr(Wq), _ptr(Wk), _ptr(Wv), _ptr(Wa), _ptr(ba), _ptr(Wb),
                                      _ptr(bb), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(o), _ptr(ws),
                                      ws.numel(), _stream(stream)))
    return dict(o=o, S=S_out, cache=cache_out)


def prefill_static_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_prefill_static_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def prefill_static(q, k, v, alpha, beta, wq, wk, wv, S0=None, cache_q=None, cache_k=None, cache_v=None, *,
                   out_dtype=torch.float32, seg_len: int | None = None, o=None, S_final=None,
                   want_cache_out=True, ws=None, stream=None, d_model: int = 128):
    """jb_prefill_static: the static-conv block.  q,k [B,T,H,dk], v [B,T,H,dv] (bf16), alpha,beta
    [B,T,H] f32, weights wq,wk [H*dk,4], wv [H*dv,4] f32, caches [B,3,H,d] (all three or none).
    Returns dict(o, S_final, cache_q, cache_k, cache_v)."""
    B, T, H, dk = q.shape
    dv = v.shape[3]
    shape = make_shape(B, T, H, dk, dv, d_model, _io_code(q), _DT[out_dtype],
                       flag_segment(seg_len) if seg_len else 0)
    dev = q.device
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    if S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    outs = [None, None, None]
    if want_cache_out:
        outs = [torch.empty((B, 3, H, d), dtype=q.dtype, device=dev) for d in (dk, dk, dv)]
    need = prefill_static_workspace_size(shape)
    if ws is None and need > 0:
        ws = workspace(need, dev)
    _check(_lib.jb_prefill_static(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                  _ptr(wq), _ptr(wk), _ptr(wv), _ptr(S0), _ptr(cache_q), _ptr(cache_k),
                                  _ptr(cache_v), _ptr(o), _ptr(S_final), _ptr(outs[0]), _ptr(outs[1]),
                                  _ptr(outs[2]), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return dict(o=o, S_final=S_final, cache_q=outs[0], cache_k=outs[1], cache_v=outs[2])


def decode_step_static(S, cache_q, cache_k, cache_v, q_t, k_t, v_t, alpha_t, beta_t, wq, wk, wv, *,
                       out_dtype=torch.float32, S_out=None, cache_q_out=None, cache_k_out=None,
                       cache_v_out=None, o=None, stream=None, d_model: int = 128):
    """jb_decode_step_static: one decode step of the static-conv block.  In place on S and the
    caches unless the *_out tensors are given.  Returns dict(o, S, cache_q, cache_k, cache_v)."""
    B, H, dk = q_t.shape
    dv = v_t.shape[2]
    shape = make_shape(B, 1, H, dk, dv, d_model, _io_code(q_t), _DT[out_dtype])
    S_out = S if S_out is None else S_out
    cq = cache_q if cache_q_out is None else cache_q_out
    ck = cache_k if cache_k_out is None else cache_k_out
    cv = cache_v if cache_v_out is None else cache_v_out
    if o is None:
        o = torch.empty((B, H, dv), dtype=out_dtype, device=q_t.device)
    _check(_lib.jb_decode_step_static(ctypes.byref(shape), _ptr(S), _ptr(S_out), _ptr(cache_q), _ptr(cache_k),
                                      _ptr(cache_v), _ptr(cq), _ptr(ck), _ptr(cv), _ptr(q_t), _ptr(k_t),
                                      _ptr(v_t), _ptr(alpha_t), _ptr(beta_t), _ptr(wq), _ptr(wk), _ptr(wv),
                                      _ptr(o), _stream(stream)))
    return dict(o=o, S=S_out, cache_q=cq, cache_k=ck, cache_v=cv)


def prefill_varlen_workspace_size(shape: Shape, total_tokens: int) -> int:
    n = _SZ(0)
    _check(_lib.jb_prefill_varlen_workspace_size(ctypes.byref(shape), int(total_tokens), ctypes.byref(n)))
    return n.value


def prefill_varlen(cu_seqlens, x, q, k, v, alpha, beta, W1, W2, b1=None, b2=None, S0=None, conv_in=None, *,
                   max_seqlen: int | None = None, out_dtype=torch.float32, seg_len: int | None = None, o=None,
                   S_final=None, conv_out=None, want_conv_out=True, ws=None, stream=None):
    """jb_prefill_varlen: B packed sequences.  cu_seqlens int32 [B+1] (device; its host copy is
    read once for the longest length unless max_seqlen is given), x [total,D], q,k [total,H,dk],
    v [total,H,dv], alpha,beta [total,H].  Returns dict(o, S_final, conv_out) with per-sequence
    S_final [B,H,dk,dv] and conv_out [B,3,H,dv]."""
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    B = cu_seqlens.numel() - 1
    total, D = x.shape
    H, dk = q.shape[1], q.shape[2]
    dv = v.shape[2]
    if max_seqlen is None:
        lens = cu_seqlens.cpu().diff()
        max_seqlen = int(lens.max()) if B > 0 else 0
    shape = make_shape(B, max_seqlen, H, dk, dv, D, _io_code(x), _DT[out_dtype],
                       flag_segment(seg_len) if seg_len else 0)
    dev = x.device
    if o is None:
        o = torch.empty((total, H, dv), dtype=out_dtype, device=dev)
    if S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if conv_out is None and want_conv_out:
        conv_out = torch.empty((B, 3, H, dv), dtype=x.dtype, device=dev)
    need = prefill_varlen_workspace_size(shape, total)
    if ws is None:
        ws = workspace(need, dev)
    _check(_lib.jb_prefill_varlen(ctypes.byref(shape), total, _ptr(cu_seqlens), _ptr(x), _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(alpha), _ptr(beta), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(S0),
                                  _ptr(conv_in), _ptr(o), _ptr(S_final), _ptr(conv_out), _ptr(ws), ws.numel(),
                                  _stream(stream)))
    return dict(o=o, S_final=S_final, conv_out=conv_out)


def backward_workspace_size(shape: Shape) -> int:
    n = _SZ(0)
    _check(_lib.jb_backward_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def backward(x, q, k, v, alpha, beta, W1, W2, dout, b1=None, b2=None, S0=None, conv_in=None, dS_final=None,
             dconv_out=None, *, ws=None, stream=None):
    """jb_backward: gradients of jb_prefill.  Returns a dict of float32 tensors dx, dq, dk, dv,
    dalpha, dbeta, dW1, db1, dW2, db2, dS0, dconv_in."""
    B, T, D = x.shape
    H, dk = q.shape[2], q.shape[3]
    dv = v.shape[3]
    shape = make_shape(B, T, H, dk, dv, D, _io_code(x), JB_F32)
    dev = x.device
    f = lambda *sz: torch.empty(sz, dtype=torch.float32, device=dev)
    out = dict(dx=f(B, T, D), dq=f(B, T, H, dk), dk=f(B, T, H, dk), dv=f(B, T, H, dv), dalpha=f(B, T, H),
               dbeta=f(B, T, H), dW1=f(32, D), db1=f(32), dW2=f(4 * H, 32), db2=f(4 * H), dS0=f(B, H, dk, dv),
               dconv_in=f(B, 3, H, dv))
    if ws is None:
        ws = workspace(backward_workspace_size(shape), dev)
    _check(_lib.jb_backward(ctypes.byref(shape), _ptr(x), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                            _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(S0), _ptr(conv_in), _ptr(dout),
                            _ptr(dS_final), _ptr(dconv_out),
                            *[_ptr(out[n]) for n in ("dx", "dq", "dk", "dv", "dalpha", "dbeta", "dW1", "db1", "dW2",
                                                     "db2", "dS0", "dconv_in")],
                            _ptr(ws), ws.numel(), _stream(stream)))
    return out


# ---------------------------------------------------------------- softmax-attention layers


def _rows(t, name: str):
    """Pointer, tokens and token stride of [..., heads, D] whose tokens lie at one distance."""
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        n, heads, d = shape
        stride = st[0]
    elif len(shape) == 4:
        B, T, heads, d = shape
        n, stride = B * T, st[1] if T > 1 else st[0]
        if B > 1 and T > 1 and st[0] != T * stride:
            raise ValueError(f"{name}: tokens must lie at one distance")
    else:
        raise ValueError(f"{name}: expected [tokens, heads, D] or [B, T, heads, D], got {tuple(shape)}")
    if st[-1] != 1 or (heads > 1 and st[-2] != d):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if n <= 1:
        return t.data_ptr(), n, 0
    if stride < heads * d:
        raise ValueError(f"{name}: tokens overlap (token stride {stride})")
    return t.data_ptr(), n, stride


def _same(di, *groups):
    """Every tensor of each (dtype, names, tensors) group of that dtype and on device di."""
    for dtype, names, tensors in groups:
        for t in tensors:
            if t is not None and (t.dtype is not dtype or t.get_device() != di):
                name = names.split()[[x is t for x in tensors].index(True)]
                if t.dtype is not dtype:
                    raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
                raise ValueError(f"{name} is on {t.device}, q on cuda:{di}")


def _flat(t, name: str, *shape):
    """Pointer of a contiguous tensor of the given shape (None: no pointer)."""
    if t is None:
        return None
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _positions(t, n: int):
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"positions: expected {n} contiguous values, got {tuple(t.shape)}")
    return t.data_ptr()


# the handle of a device's current stream (the public accessor builds a Stream object, 2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda di: torch.cuda.current_stream(di).cuda_stream)


def _device(q) -> int:
    if not q.is_cuda:
        raise ValueError("libjetblock takes device tensors; got a tensor on " + str(q.device))
    return q.get_device()


def _launch(di: int, fn, *args):
    """fn(*args, stream) on device di's current stream."""
    if di == torch.cuda.current_device():
        _check(fn(*args, _raw_stream(di)))
    else:
        with torch.cuda.device(di):
            _check(fn(*args, _raw_stream(di)))


def _on_stream(fn, args):
    """fn(**args) on the stream args names (a torch stream or a handle): the call, and what it
    allocates, belong to that stream, so nothing it still uses is handed out on another."""
    args = dict(args)
    stream, di = args.pop("stream"), _device(args["q"])
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=args["q"].device)
    elif stream.device.index != di:
        raise ValueError(f"stream is of {stream.device}, q on cuda:{di}")
    with torch.cuda.stream(stream):
        return fn(**args)


def _empty(like, dtype):
    """An uninitialised contiguous tensor of `like`'s shape and device."""
    if dtype is like.dtype and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=dtype, device=like.device)


def _rope_flags(interleaved, normalize):
    return (ROPE_INTERLEAVED if interleaved else 0) | (0 if normalize else ROPE_NO_NORM)


def qk_norm_rope(q, k, positions, inv_freq, wq=None, wk=None, *, eps=1e-6, interleaved=False, normalize=True,
                 out_dtype=None, q_out=None, k_out=None, stream=None):
    """jb_qk_norm_rope.  q [tokens,H,D] or [B,T,H,D], k likewise with Hkv heads (any distance
    between tokens), positions int32 [tokens], inv_freq f32 [rot/2], wq, wk [D].  Returns
    (q_out, k_out), contiguous, of out_dtype (default: q's)."""
    if stream is not None:
        return _on_stream(qk_norm_rope, locals())
    di, io = _device(q), q.dtype
    out_dtype = out_dtype or (q_out.dtype if q_out is not None else io)
    _same(di, (io, "k wq wk", (k, wq, wk)), (torch.int32, "positions", (positions,)),
          (torch.float32, "inv_freq", (inv_freq,)), (out_dtype, "q_out k_out", (q_out, k_out)))
    H, D = q.shape[-2:]
    Hkv, pairs = k.shape[-2], inv_freq.numel()
    qp, n, qs = _rows(q, "q")
    kp, nk, ks = _rows(k, "k")
    if nk != n or k.shape[-1] != D:
        raise ValueError(f"k {tuple(k.shape)} does not go with q {tuple(q.shape)}")
    if q_out is None:
        q_out = _empty(q, out_dtype)
    if k_out is None:
        k_out = _empty(k, out_dtype)
    shape = AttnShape(1, n, H, Hkv, D, 2 * pairs, 0, 0, 0, 0, 0, _io_code(q), _code(out_dtype),
                      _rope_flags(interleaved, normalize), qs, ks, 0, 0)
    _launch(di, _lib.jb_qk_norm_rope, shape, qp, kp, _flat(wq, "wq", D), _flat(wk, "wk", D),
            _flat(inv_freq, "inv_freq", pairs), _positions(positions, n), eps,
            _flat(q_out, "q_out", *q.shape), _flat(k_out, "k_out", *k.shape))
    return q_out, k_out


def qk_norm_rope_backward_workspace_size(shape: AttnShape) -> int:
    n = _SZ(0)
    _check(_lib.jb_qk_norm_rope_backward_workspace_size(shape, n))
    return n.value


def qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, wq=None, wk=None, *, eps=1e-6,
                          interleaved=False, normalize=True, dq=None, dk=None, ws=None, stream=None):
    """jb_qk_norm_rope_backward: gradients of qk_norm_rope from those of its outputs (contiguous,
    bf16 or f32).  Returns dict(dq, dk, dwq, dwk): dq, dk of dq_out's dtype, dwq, dwk f32 [D]
    (None without the norm)."""
    if stream is not None:
        return _on_stream(qk_norm_rope_backward, locals())
    di, dev, io, gr = _device(q), q.device, q.dtype, dq_out.dtype
    _same(di, (io, "k wq wk", (k, wq, wk)), (torch.int32, "positions", (positions,)),
          (torch.float32, "inv_freq", (inv_freq,)), (gr, "dq_out dk_out dq dk", (dq_out, dk_out, dq, dk)),
          (torch.uint8, "ws", (ws,)))
    H, D = q.shape[-2:]
    Hkv, pairs = k.shape[-2], inv_freq.numel()
    qp, n, qs = _rows(q, "q")
    kp, nk, ks = _rows(k, "k")
    if nk != n or k.shape[-1] != D:
        raise ValueError(f"k {tuple(k.shape)} does not go with q {tuple(q.shape)}")
    dq = _empty(q, gr) if dq is None else dq
    dk = _empty(k, gr) if dk is None else dk
    dwq = dwk = None
    if normalize:
        dwq = torch.empty(D, dtype=torch.float32, device=dev)
        dwk = torch.empty(D, dtype=torch.float32, device=dev)
    shape = AttnShape(1, n, H, Hkv, D, 2 * pairs, 0, 0, 0, 0, 0, _io_code(q), _code(gr),
                      _rope_flags(interleaved, normalize), qs, ks, 0, 0)
    if ws is None:
        ws = workspace(qk_norm_rope_backward_workspace_size(shape), dev)
    _launch(di, _lib.jb_qk_norm_rope_backward, shape, qp, kp, _flat(wq, "wq", D), _flat(wk, "wk", D),
            _flat(inv_freq, "inv_freq", pairs), _positions(positions, n), eps,
            _flat(dq_out, "dq_out", *q.shape), _flat(dk_out, "dk_out", *k.shape), _flat(dq, "dq", *q.shape),
            _flat(dk, "dk", *k.shape), _flat(dwq, "dwq", D), _flat(dwk, "dwk", D), ws.data_ptr(), ws.numel())
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _batch(q, cu_seqlens, max_seqlen):
    """B and T of q: packed [tokens,H,D] with cu_seqlens, [B,T,H,D], or [B,H,D] (one token each).
    Packed rows that no sequence owns may be more than B max_seqlen has room for: T covers them."""
    if cu_seqlens is not None:
        if q.dim() != 3 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("packed: q is [tokens, H, D] and cu_seqlens [B + 1]")
        B, n = cu_seqlens.numel() - 1, q.shape[0]
        if max_seqlen is not None and max_seqlen < 0:
            raise ValueError(f"max_seqlen = {max_seqlen} must be >= 0")
        return B, n if max_seqlen is None else min(max(int(max_seqlen), -(-n // B)), n)
    return (q.shape[0], q.shape[1]) if q.dim() == 4 else (q.shape[0], 1)


def _pages(k_cache, v_cache, page_table, kv_lens, B, D):
    """num_pages, Hkv, page, page stride and max_pages of a cache."""
    shape, st = k_cache.shape, k_cache.stride()
    vst = v_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or \
            vst != st and any(n > 1 and a != b for n, a, b in zip(shape, st, vst)):
        raise ValueError("k_cache and v_cache are [pages, Hkv, page, D] alike")
    P, Hkv, page, d = shape
    if d != D or st[3] != 1 or st[2] != D or (Hkv > 1 and st[1] != page * D):
        raise ValueError("a page of the caches must be contiguous, of q's head size")
    table = page_table.shape
    if len(table) != 2 or table[0] != B:
        raise ValueError(f"page_table: expected [{B}, max_pages], got {tuple(table)}")
    if kv_lens.shape != (B,):
        raise ValueError(f"kv_lens: expected [{B}], got {tuple(kv_lens.shape)}")
    if P > 1 and st[0] < Hkv * page * D:
        raise ValueError(f"pages of the caches overlap (page stride {st[0]})")
    return P, Hkv, page, st[0] if P > 1 else 0, table[1]


def qk_norm_rope_paged(q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq, wq=None, wk=None, *,
                       cu_seqlens=None, max_seqlen: int | None = None, positions=None, eps=1e-6, interleaved=False,
                       normalize=True, q_out=None, stream=None):
    """jb_qk_norm_rope_paged: rotated queries out, rotated keys and values into the caches
    [pages,Hkv,page,D] (in place).  q [B,T,H,D], [B,H,D] (one token each) or packed [tokens,H,D]
    with cu_seqlens int32 [B+1]; page_table int32 [B,max_pages], kv_lens int32 [B] (the new tokens
    among the rows).  max_seqlen (packed) is a limit: of a longer sequence the tokens behind its
    first max_seqlen may be left out, neither appended nor written to q's output (default: none
    are).  Returns dict(q, k_cache, v_cache)."""
    if stream is not None:
        return _on_stream(qk_norm_rope_paged, locals())
    di, io = _device(q), q.dtype
    _same(di, (io, "k v k_cache v_cache wq wk q_out", (k, v, k_cache, v_cache, wq, wk, q_out)),
          (torch.int32, "page_table kv_lens cu_seqlens positions", (page_table, kv_lens, cu_seqlens, positions)),
          (torch.float32, "inv_freq", (inv_freq,)))
    H, D = q.shape[-2:]
    pairs = inv_freq.numel()
    qp, n, qs = _rows(q, "q")
    kp, nk, ks = _rows(k, "k")
    vp, nv, vs = _rows(v, "v")
    B, T = _batch(q, cu_seqlens, max_seqlen)
    P, Hkv, page, ps, max_pages = _pages(k_cache, v_cache, page_table, kv_lens, B, D)
    if nk != n or nv != n or k.shape[-2:] != (Hkv, D) or v.shape[-2:] != (Hkv, D):
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not go with q {tuple(q.shape)} and the caches")
    if q_out is None:
        q_out = _empty(q, io)
    code = _io_code(q)
    shape = AttnShape(B, T, H, Hkv, D, 2 * pairs, page, max_pages, P, 0, 0, code, code,
                      _rope_flags(interleaved, normalize), qs, ks, vs, ps)
    _launch(di, _lib.jb_qk_norm_rope_paged, shape, n,
            None if cu_seqlens is None else _flat(cu_seqlens, "cu_seqlens", B + 1), _flat(kv_lens, "kv_lens", B),
            _flat(page_table, "page_table", B, max_pages), qp, kp, vp, _flat(wq, "wq", D), _flat(wk, "wk", D),
            _flat(inv_freq, "inv_freq", pairs),
            None if positions is None else _positions(positions, n), eps,
            _flat(q_out, "q_out", *q.shape), k_cache.data_ptr(), v_cache.data_ptr())
    return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache}


def attn_paged_workspace_size(shape: AttnShape, total_tokens: int, packed: bool) -> int:
    n = _SZ(0)
    _check(_lib.jb_attn_paged_workspace_size(shape, int(total_tokens), int(packed), n))
    return n.value


def attn_paged(q, k_cache, v_cache, page_table, kv_lens, *, cu_seqlens=None, max_seqlen: int | None = None,
               max_kv: int | None = None, window: int = 0, scale: float | None = None, out_dtype=None, o=None,
               want_lse=False, lse=None, ws=None, stream=None):
    """jb_attn_paged: attention of each sequence's new tokens over its paged cache (which holds
    them already).  q [B,T,H,D], [B,H,D] (decode) or packed [tokens,H,D] with cu_seqlens int32
    [B+1]; caches, page_table and kv_lens as for qk_norm_rope_paged.  max_seqlen and max_kv, host
    integers, are the longest sequence's new tokens (packed; default: all) and cache rows (default:
    the table's capacity); the launch is planned by them, nothing is read back from the device.
    max_kv is a hint, longer caches are right too; max_seqlen is a limit: of a longer sequence the
    tokens behind its first max_seqlen may be left out, their rows of o and lse not written.  scale
    None (or 0) is 1 / sqrt(D).  Returns dict(o, lse): o of q's shape and out_dtype (default: q's;
    float32 also takes the softmax weights more exactly), lse f32 [..., H] or None."""
    if stream is not None:
        return _on_stream(attn_paged, locals())
    di, io = _device(q), q.dtype
    out_dtype = out_dtype or (o.dtype if o is not None else io)
    _same(di, (io, "k_cache v_cache", (k_cache, v_cache)),
          (torch.int32, "page_table kv_lens cu_seqlens", (page_table, kv_lens, cu_seqlens)),
          (out_dtype, "o", (o,)), (torch.float32, "lse", (lse,)), (torch.uint8, "ws", (ws,)))
    H, D = q.shape[-2:]
    qp, n, qs = _rows(q, "q")
    B, T = _batch(q, cu_seqlens, max_seqlen)
    P, Hkv, page, ps, max_pages = _pages(k_cache, v_cache, page_table, kv_lens, B, D)
    if not 0 <= window <= 1 << 30:
        raise ValueError(f"window = {window} not in [0, 2^30]")
    max_kv = 0 if max_kv is None else max(1, min(int(max_kv), max_pages * page))
    if o is None:
        o = _empty(q, out_dtype)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    packed = cu_seqlens is not None
    shape = AttnShape(B, T, H, Hkv, D, 0, page, max_pages, P, max_kv, int(window),
                      _io_code(q), _code(out_dtype), 0, qs, 0, 0, ps)
    if ws is None:
        need = attn_paged_workspace_size(shape, n, packed)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _launch(di, _lib.jb_attn_paged, shape, n, _flat(cu_seqlens, "cu_seqlens", B + 1),
            _flat(kv_lens, "kv_lens", B), _flat(page_table, "page_table", B, max_pages), qp, k_cache.data_ptr(),
            v_cache.data_ptr(), 0.0 if scale is None else float(scale), _flat(o, "o", *q.shape),
            _flat(lse, "lse", *q.shape[:-1]), None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel())
    return {"o": o, "lse": lse}
