"""Python binding of librglru.so (include/rglru.h): argument marshalling only.

Each function takes torch tensors, checks dtype / device / contiguity, passes raw device pointers
and the current HIP stream to the C entry point of the same name, and raises RglruError on a
non-zero status. Every step of the computation runs in the library's HIP kernels; there is no
fallback of any kind: if librglru.so is missing or fails to load, importing this package fails. The local
attention block's operators go through a second module, _rglru_torch.so, built against this interpreter's
torch; if that is missing, they raise ImportError and the recurrent block's work without it.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librglru.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run gated_linear_recurrence_conv1d_amd/build.py "
                      "(or __graft_entry__.build())")
_lib = ctypes.CDLL(LIB_PATH)


class _NotThere:
    """Stands where the module _rglru_torch should be: any use of it says what is missing."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError("_rglru_torch.so, which the attention block's operators need, is not built or does not "
                          "load; run gated_linear_recurrence_conv1d_amd/build.py (or __graft_entry__.build())"
                          ) from self._why


try:
    from . import _rglru_torch as _ext  # checks and calls of the attention block's operators
except ImportError as e:  # the recurrent block's operators need none of it
    _ext = _NotThere(e)

RGLRU_OK = 0
RGLRU_ERR_INVALID_ARG = 1
RGLRU_ERR_UNSUPPORTED = 2
RGLRU_ERR_WORKSPACE = 3
RGLRU_ERR_HIP = 4
RGLRU_F32 = 0
RGLRU_BF16 = 1
RGLRU_PLAN_AUTO = 0
RGLRU_PLAN_DIRECT = 1
RGLRU_PLAN_CHUNKED = 2
RGLRU_PLAN_FUSED = 3
_PLANS = {"auto": RGLRU_PLAN_AUTO, "direct": RGLRU_PLAN_DIRECT, "chunked": RGLRU_PLAN_CHUNKED,
          "fused": RGLRU_PLAN_FUSED}

_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_lib.rglru_status_string.argtypes = [_i]
_lib.rglru_status_string.restype = ctypes.c_char_p
_lib.rglru_forward_workspace_size.argtypes = [_i] * 5
_lib.rglru_forward_workspace_size.restype = _sz
_lib.rglru_scan_workspace_size.argtypes = [_i] * 5
_lib.rglru_scan_workspace_size.restype = _sz
_lib.rglru_forward_workspace_size_planned.argtypes = [_i] * 7
_lib.rglru_forward_workspace_size_planned.restype = _sz
_lib.rglru_lookback_failures.argtypes = [_vp, _sz, ctypes.POINTER(ctypes.c_uint), _vp]
_lib.rglru_lookback_failures.restype = _i
_lib.rglru_forward_plan_info.argtypes = [_i] * 5 + [ctypes.POINTER(_i), ctypes.POINTER(_i)]
_lib.rglru_forward_plan_info.restype = _i
_lib.rglru_forward.argtypes = [_vp] * 10 + [_i] * 5 + [_vp, _sz, _vp]
_lib.rglru_forward.restype = _i
_lib.rglru_forward_noalloc.argtypes = [_vp] * 10 + [_i] * 5 + [_vp]
_lib.rglru_forward_noalloc.restype = _i
_lib.rglru_forward_noalloc_max_bytes.argtypes = []
_lib.rglru_forward_noalloc_max_bytes.restype = _sz
_lib.rglru_forward_planned.argtypes = [_vp] * 10 + [_i] * 5 + [_vp, _sz, _vp, _i, _i]
_lib.rglru_forward_planned.restype = _i
_lib.rglru_gate_preacts.argtypes = [_vp] * 7 + [_i] * 5 + [_vp]
_lib.rglru_gate_preacts.restype = _i
_lib.rglru_scan_preacts.argtypes = [_vp] * 7 + [_i] * 5 + [_vp, _sz, _vp, _i, _i]
_lib.rglru_scan_preacts.restype = _i
_lib.rglru_decode_step.argtypes = [_vp] * 10 + [_i] * 4 + [_vp]
_lib.rglru_decode_step.restype = _i
_lib.rglru_prefill_state.argtypes = [_vp, _vp] + [_i] * 4 + [_vp]
_lib.rglru_prefill_state.restype = _i
_lib.rglru_local_mqa.argtypes = [_vp] * 4 + [_i] * 5 + [ctypes.c_float, _i, _vp]
_lib.rglru_local_mqa.restype = _i
_lib.rglru_backward_workspace_size.argtypes = [_i] * 5
_lib.rglru_backward_workspace_size.restype = _sz
_lib.rglru_backward.argtypes = [_vp] * 19 + [_i] * 5 + [_vp, _sz, _vp]
_lib.rglru_backward.restype = _i
_ll = ctypes.c_longlong
_f = ctypes.c_float
_lib.rglru_qk_norm_rope.argtypes = [_vp] * 12 + [_i] * 5 + [_ll] * 6 + [_f, _i, _vp]
_lib.rglru_qk_norm_rope.restype = _i
_lib.rglru_qk_norm_rope_backward_workspace_size.argtypes = [_i, _i]
_lib.rglru_qk_norm_rope_backward_workspace_size.restype = _sz
_lib.rglru_qk_norm_rope_backward.argtypes = ([_vp] * 12 + [_i] * 5 + [_ll] * 6 +
                                             [_f, _i, _vp, _sz, _vp])
_lib.rglru_qk_norm_rope_backward.restype = _i
_lib.rglru_local_attention.argtypes = [_vp] * 6 + [_i] * 5 + [_ll] * 3 + [_i, _i, _f, _i, _vp]
_lib.rglru_local_attention.restype = _i
_lib.rglru_local_attention_backward_workspace_size.argtypes = [_i] * 7
_lib.rglru_local_attention_backward_workspace_size.restype = _sz
_lib.rglru_local_attention_backward.argtypes = ([_vp] * 10 + [_i] * 5 + [_ll] * 6 +
                                                [_i, _i, _f, _i, _vp, _sz, _vp])
_lib.rglru_local_attention_backward.restype = _i
_lib.rglru_paged_attention_workspace_size.argtypes = [_i] * 9
_lib.rglru_paged_attention_workspace_size.restype = _sz
_lib.rglru_paged_attention.argtypes = ([_vp] * 6 + [_i] * 4 + [_ll] + [_i] * 5 +
                                       [_f, _i, _vp, _sz, _vp])
_lib.rglru_paged_attention.restype = _i


class RglruError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {rglru_status_string(status)} (status {status})")
        self.status = status


def rglru_status_string(status: int) -> str:
    return _lib.rglru_status_string(int(status)).decode()


def _dt(dtype) -> int:
    if dtype in (torch.bfloat16, "bf16", RGLRU_BF16):
        return RGLRU_BF16
    if dtype in (torch.float32, "f32", RGLRU_F32):
        return RGLRU_F32
    raise ValueError(f"unsupported dtype {dtype}")


def _ptr(t, io_dtype=None, name=""):
    """Raw device pointer of a contiguous CUDA (HIP) tensor, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if io_dtype is not None and t.dtype != io_dtype:
        raise ValueError(f"{name}: expected {io_dtype}, got {t.dtype}")
    return t.data_ptr()


def _shape(t, shape, name):
    """Raise ValueError unless tensor t (if given) has exactly this shape. Every buffer's size is
    checked here, before any call: the C ABI takes sizes only through B, T, D, H, N, so a tensor
    of another size would be read or written out of its bounds on the device."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _dims(x, W_a):
    if x.dim() != 3:
        raise ValueError(f"x: expected [B, T, D], got shape {tuple(x.shape)}")
    B, T, D = x.shape
    if W_a.dim() != 3 or W_a.shape[0] < 1 or D % W_a.shape[0]:
        raise ValueError(f"W_a: expected [H, D/H, D/H] with D = {D}, got {tuple(W_a.shape)}")
    return B, T, D, W_a.shape[0]


def _check_params(D, H, conv_w, W_a, b_a, W_x, b_x, Lam):
    Dh = D // H
    _shape(conv_w, (4, D), "conv_w")
    _shape(W_a, (H, Dh, Dh), "W_a")
    _shape(W_x, (H, Dh, Dh), "W_x")
    _shape(b_a, (D,), "b_a")
    _shape(b_x, (D,), "b_x")
    _shape(Lam, (D,), "Lambda")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _as_stream(stream, t):
    """A stream of t's device, or its number, as a torch stream."""
    index = t.get_device()
    if not isinstance(stream, torch.cuda.Stream):
        return (torch.cuda.ExternalStream(int(stream), device=index) if int(stream) else
                torch.cuda.default_stream(index))  # (0 would be a new one)
    if stream.device_index != index:
        raise ValueError(f"stream: on {stream.device}, expected {t.device}")
    return stream


def _on(stream, t, f):
    """f() with `stream` current, so that what f allocates comes from that stream's pool: a block of the pool of
    the stream that is current now may still be in use there, by work queued before it was freed. The results
    are recorded on the one that is current now, where the caller may use them."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return f()  # refused there
    stream, here = _as_stream(stream, t), torch.cuda.current_stream(t.device)
    with torch.cuda.stream(stream):
        out = f()
    if stream != here:
        for x in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
            if x is not None:
                x.record_stream(here)
    return out


def _check(status, where):
    if status != RGLRU_OK:
        raise RglruError(status, where)


def rglru_forward_workspace_size(B, T, D, H, dtype) -> int:
    return int(_lib.rglru_forward_workspace_size(B, T, D, H, _dt(dtype)))


def rglru_scan_workspace_size(B, T, D, H, dtype) -> int:
    return int(_lib.rglru_scan_workspace_size(B, T, D, H, _dt(dtype)))


def rglru_forward_workspace_size_planned(B, T, D, H, dtype, plan="auto", chunk_len=0) -> int:
    return int(_lib.rglru_forward_workspace_size_planned(B, T, D, H, _dt(dtype), _PLANS[plan],
                                                         int(chunk_len)))


def rglru_lookback_failures(workspace, stream=None) -> int:
    """Look-back waits of the last forward / backward call on `workspace` that gave up (0 after
    a normal call). Waits for the stream."""
    n = ctypes.c_uint(0)
    _check(_lib.rglru_lookback_failures(_ptr(workspace, None, "workspace"),
                                        workspace.numel() * workspace.element_size(),
                                        ctypes.byref(n), _stream(stream)),
           "rglru_lookback_failures")
    return int(n.value)


def rglru_forward_plan_info(B, T, D, H, dtype):
    plan, chunk = _i(), _i()
    _check(_lib.rglru_forward_plan_info(B, T, D, H, _dt(dtype), ctypes.byref(plan),
                                        ctypes.byref(chunk)), "rglru_forward_plan_info")
    return {RGLRU_PLAN_DIRECT: "direct", RGLRU_PLAN_CHUNKED: "chunked",
            RGLRU_PLAN_FUSED: "fused"}[plan.value], chunk.value


def _fwd_args(x, conv_w, W_a, b_a, W_x, b_x, Lam, h0, y, h_T):
    io = x.dtype
    B, T, D, H = _dims(x, W_a)
    _check_params(D, H, conv_w, W_a, b_a, W_x, b_x, Lam)
    _shape(h0, (B, D), "h0")
    _shape(y, (B, T, D), "y")
    _shape(h_T, (B, D), "h_T")
    f32 = torch.float32
    ptrs = [_ptr(x, io, "x"), _ptr(conv_w, io, "conv_w"), _ptr(W_a, io, "W_a"),
            _ptr(b_a, f32, "b_a"), _ptr(W_x, io, "W_x"), _ptr(b_x, f32, "b_x"),
            _ptr(Lam, f32, "Lambda"), _ptr(h0, f32, "h0"), _ptr(y, io, "y"),
            _ptr(h_T, f32, "h_T")]
    return ptrs, (B, T, D, H, _dt(io))


def rglru_forward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T, workspace, stream=None):
    ptrs, dims = _fwd_args(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T)
    _check(_lib.rglru_forward(*ptrs, *dims, _ptr(workspace, None, "workspace"),
                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "rglru_forward")


def rglru_forward_noalloc(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T, stream=None):
    """rglru_forward with the library's own fixed device workspace (no allocation)."""
    ptrs, dims = _fwd_args(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T)
    _check(_lib.rglru_forward_noalloc(*ptrs, *dims, _stream(stream)), "rglru_forward_noalloc")


def rglru_forward_noalloc_max_bytes() -> int:
    return int(_lib.rglru_forward_noalloc_max_bytes())


def rglru_forward_planned(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T, workspace,
                          plan="auto", chunk_len=0, stream=None):
    ptrs, dims = _fwd_args(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T)
    _check(_lib.rglru_forward_planned(*ptrs, *dims, _ptr(workspace, None, "workspace"),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream), _PLANS[plan], int(chunk_len)),
           "rglru_forward_planned")


def rglru_gate_preacts(x, conv_w, W_a, b_a, W_x, b_x, pre, stream=None):
    """pre: int32 [B,T,D] (fp16 pairs) for bf16 x, float32 [B,T,D,2] for fp32 x."""
    io = x.dtype
    B, T, D, H = _dims(x, W_a)
    _check_params(D, H, conv_w, W_a, b_a, W_x, b_x, None)
    _check_pre(pre, x)
    f32 = torch.float32
    _check(_lib.rglru_gate_preacts(_ptr(x, io, "x"), _ptr(conv_w, io, "conv_w"),
                                   _ptr(W_a, io, "W_a"), _ptr(b_a, f32, "b_a"),
                                   _ptr(W_x, io, "W_x"), _ptr(b_x, f32, "b_x"),
                                   _ptr(pre, None, "pre"), B, T, D, H, _dt(io), _stream(stream)),
           "rglru_gate_preacts")


def _check_pre(pre, x):
    B, T, D = x.shape
    if x.dtype == torch.bfloat16:
        _shape(pre, (B, T, D), "pre")
        if pre.dtype != torch.int32:
            raise ValueError("pre: expected int32 (fp16 pairs) for bf16 x")
    else:
        _shape(pre, (B, T, D, 2), "pre")
        if pre.dtype != torch.float32:
            raise ValueError("pre: expected float32 pairs for fp32 x")


def rglru_scan_preacts(x, pre, conv_w, Lambda, h0, y, h_T, H, workspace=None, plan="auto",
                       chunk_len=0, stream=None):
    io = x.dtype
    if x.dim() != 3:
        raise ValueError(f"x: expected [B, T, D], got shape {tuple(x.shape)}")
    B, T, D = x.shape
    if H < 1 or D % H:
        raise ValueError(f"H = {H} must divide D = {D}")
    _check_pre(pre, x)
    _shape(conv_w, (4, D), "conv_w")
    _shape(Lambda, (D,), "Lambda")
    _shape(h0, (B, D), "h0")
    _shape(y, (B, T, D), "y")
    _shape(h_T, (B, D), "h_T")
    f32 = torch.float32
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rglru_scan_preacts(_ptr(x, io, "x"), _ptr(pre, None, "pre"),
                                   _ptr(conv_w, io, "conv_w"), _ptr(Lambda, f32, "Lambda"),
                                   _ptr(h0, f32, "h0"), _ptr(y, io, "y"), _ptr(h_T, f32, "h_T"),
                                   B, T, D, H, _dt(io), _ptr(workspace, None, "workspace"), wsb,
                                   _stream(stream), _PLANS[plan], int(chunk_len)),
           "rglru_scan_preacts")


def rglru_decode_step(x_t, conv_state, h, y_t, conv_w, W_a, b_a, W_x, b_x, Lambda, stream=None):
    io = x_t.dtype
    if x_t.dim() != 2:
        raise ValueError(f"x_t: expected [N, D], got shape {tuple(x_t.shape)}")
    N, D = x_t.shape
    if W_a.dim() != 3 or W_a.shape[0] < 1 or D % W_a.shape[0]:
        raise ValueError(f"W_a: expected [H, D/H, D/H] with D = {D}, got {tuple(W_a.shape)}")
    H = W_a.shape[0]
    _check_params(D, H, conv_w, W_a, b_a, W_x, b_x, Lambda)
    _shape(conv_state, (N, 3, D), "conv_state")
    _shape(h, (N, D), "h")
    _shape(y_t, (N, D), "y_t")
    f32 = torch.float32
    _check(_lib.rglru_decode_step(_ptr(x_t, io, "x_t"), _ptr(conv_state, io, "conv_state"),
                                  _ptr(h, f32, "h"), _ptr(y_t, io, "y_t"),
                                  _ptr(conv_w, io, "conv_w"), _ptr(W_a, io, "W_a"),
                                  _ptr(b_a, f32, "b_a"), _ptr(W_x, io, "W_x"),
                                  _ptr(b_x, f32, "b_x"), _ptr(Lambda, f32, "Lambda"), N, D, H,
                                  _dt(io), _stream(stream)),
           "rglru_decode_step")


def rglru_prefill_state(x, conv_state, stream=None):
    """conv_state [B,3,D] (x's dtype) = the last three inputs of each sequence of x [B,T,D]."""
    io = x.dtype
    if x.dim() != 3:
        raise ValueError(f"x: expected [B, T, D], got shape {tuple(x.shape)}")
    B, T, D = x.shape
    _shape(conv_state, (B, 3, D), "conv_state")
    _check(_lib.rglru_prefill_state(_ptr(x, io, "x"), _ptr(conv_state, io, "conv_state"), B, T, D,
                                    _dt(io), _stream(stream)), "rglru_prefill_state")


def prefill_state(x, stream=None):
    """A new conv-state tensor [B,3,D] for continuing x [B,T,D] with decode steps."""
    if stream is not None:
        return _on(stream, x, lambda: prefill_state(x))
    B, T, D = x.shape
    cs = torch.empty((B, 3, D), dtype=x.dtype, device=x.device)
    rglru_prefill_state(x, cs)
    return cs


def rglru_local_mqa(q, k, v, o, window, scale=0.0, stream=None):
    """q, o [B,T,Hq,dh]; k, v [B,T,dh]; bf16."""
    if q.dim() != 4:
        raise ValueError(f"q: expected [B, T, Hq, dh], got shape {tuple(q.shape)}")
    B, T, Hq, dh = q.shape
    _shape(k, (B, T, dh), "k")
    _shape(v, (B, T, dh), "v")
    _shape(o, (B, T, Hq, dh), "o")
    bf = torch.bfloat16
    _check(_lib.rglru_local_mqa(_ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
                                _ptr(o, bf, "o"), B, T, Hq, dh, int(window), float(scale),
                                RGLRU_BF16, _stream(stream)), "rglru_local_mqa")


def local_mqa(q, k, v, window, scale=0.0, stream=None):
    """Returns o [B,T,Hq,dh] (bf16)."""
    if stream is not None:
        return _on(stream, q, lambda: local_mqa(q, k, v, window, scale))
    o = torch.empty_like(q)
    rglru_local_mqa(q, k, v, o, window, scale)
    return o


def rglru_backward_workspace_size(B, T, D, H, dtype) -> int:
    return int(_lib.rglru_backward_workspace_size(B, T, D, H, _dt(dtype)))


def rglru_backward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, dy, dh_T, dx, dconv_w, dW_a,
                   db_a, dW_x, db_x, dLambda, dh0, workspace, stream=None):
    io = x.dtype
    B, T, D, H = _dims(x, W_a)
    Dh = D // H
    _check_params(D, H, conv_w, W_a, b_a, W_x, b_x, Lambda)
    for t, shape, name in ((h0, (B, D), "h0"), (y, (B, T, D), "y"), (dy, (B, T, D), "dy"),
                           (dh_T, (B, D), "dh_T"), (dx, (B, T, D), "dx"),
                           (dconv_w, (4, D), "dconv_w"), (dW_a, (H, Dh, Dh), "dW_a"),
                           (db_a, (D,), "db_a"), (dW_x, (H, Dh, Dh), "dW_x"), (db_x, (D,), "db_x"),
                           (dLambda, (D,), "dLambda"), (dh0, (B, D), "dh0")):
        _shape(t, shape, name)
    f32 = torch.float32
    ptrs = [_ptr(x, io, "x"), _ptr(conv_w, io, "conv_w"), _ptr(W_a, io, "W_a"),
            _ptr(b_a, f32, "b_a"), _ptr(W_x, io, "W_x"), _ptr(b_x, f32, "b_x"),
            _ptr(Lambda, f32, "Lambda"), _ptr(h0, f32, "h0"), _ptr(y, io, "y"),
            _ptr(dy, io, "dy"), _ptr(dh_T, f32, "dh_T"), _ptr(dx, io, "dx"),
            _ptr(dconv_w, f32, "dconv_w"), _ptr(dW_a, f32, "dW_a"), _ptr(db_a, f32, "db_a"),
            _ptr(dW_x, f32, "dW_x"), _ptr(db_x, f32, "db_x"), _ptr(dLambda, f32, "dLambda"),
            _ptr(dh0, f32, "dh0")]
    _check(_lib.rglru_backward(*ptrs, B, T, D, H, _dt(io), _ptr(workspace, None, "workspace"),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "rglru_backward")


# ---- the local attention block's operators. Tensors of heads are [..., H, dh] with the heads of a
# token contiguous and one stride from token to token, so slices of a packed projection need no
# copy. All tensors of a call live on one device, which need not be the current one; the call runs on
# `stream` (a torch stream or a stream's number), else on that device's current stream. What a call makes
# belongs to the stream it runs on, and may be used on the one that was current, once that waits for it; the
# tensors it is given have to be ready on that stream, and to live until it is done with them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(where, fn, q, stream, *args):
    """fn(*args, stream), which checks its tensors (csrc/rglru_torch.cpp), on q's device."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q: expected a torch.Tensor")
    index = q.get_device()
    if index < 0:
        status = fn(*args, 0)  # refused there, by what is wrong with the tensors
    else:
        s = _raw_stream(index) if stream is None else _as_stream(stream, q).cuda_stream
        if index == _current_device():  # a tensor lives there: the runtime is up
            status = fn(*args, s)
        else:
            with torch.cuda.device(index):
                status = fn(*args, s)
    if status != RGLRU_OK:
        raise RglruError(status, where)


def _int32(n):
    n = int(n)
    return n if n < 0x7FFFFFFF else 0x7FFFFFFF


def rglru_qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_w=None, k_w=None, eps=1e-6,
                       v=None, k_pages=None, v_pages=None, slots=None, stream=None):
    """q [..., Hq, dh], k, v [..., Hkv, dh]; positions int32 and slots int64 [...]; inv_freq f32
    [rot / 2]; k_pages, v_pages [pages, page, Hkv, dh]. k_out may be None with slots."""
    _call("rglru_qk_norm_rope", _ext.qk_norm_rope, q, stream, q, k, v, q_w, k_w, inv_freq,
          positions, slots, q_out, k_out, k_pages, v_pages, eps)


def qk_norm_rope(q, k, positions, inv_freq, q_w=None, k_w=None, eps=1e-6, v=None, k_pages=None,
                 v_pages=None, slots=None, q_out=None, k_out=None, stream=None):
    """Returns (q_out, k_out), new contiguous tensors unless given (q and k themselves: in place)."""
    if stream is not None:
        return _on(stream, q, lambda: qk_norm_rope(q, k, positions, inv_freq, q_w, k_w, eps, v, k_pages,
                                                   v_pages, slots, q_out, k_out))
    q_out = _ext.empty_as(q) if q_out is None else q_out
    k_out = _ext.empty_as(k) if k_out is None else k_out
    rglru_qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_w, k_w, eps, v, k_pages, v_pages,
                       slots)
    return q_out, k_out


def rglru_qk_norm_rope_backward_workspace_size(rows, dh) -> int:
    return int(_lib.rglru_qk_norm_rope_backward_workspace_size(rows, dh))


def rglru_qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, dq, dk, q_w=None,
                                k_w=None, dq_w=None, dk_w=None, eps=1e-6, workspace=None,
                                stream=None):
    _call("rglru_qk_norm_rope_backward", _ext.qk_norm_rope_backward, q, stream, q, k, q_w, k_w, inv_freq,
          positions, dq_out, dk_out, dq, dk, dq_w, dk_w, eps, workspace)


def qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, q_w=None, k_w=None, eps=1e-6,
                          dq=None, dk=None, workspace=None, stream=None):
    """Returns a dict with dq, dk (new contiguous tensors unless given) and fp32 dq_w, dk_w [dh]
    (None without weights)."""
    if stream is not None:
        return _on(stream, q, lambda: qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, q_w,
                                                            k_w, eps, dq, dk, workspace))
    dev, dh = q.device, q.shape[-1]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    dq = empty(q.shape, q.dtype) if dq is None else dq
    dk = empty(k.shape, k.dtype) if dk is None else dk
    dq_w = dk_w = None
    if q_w is not None:
        dq_w, dk_w = empty((dh,), torch.float32), empty((dh,), torch.float32)
        if workspace is None:
            workspace = empty((rglru_qk_norm_rope_backward_workspace_size(positions.numel(), dh),),
                              torch.uint8)
    rglru_qk_norm_rope_backward(q, k, positions, inv_freq, dq_out, dk_out, dq, dk, q_w, k_w, dq_w,
                                dk_w, eps, workspace)
    return {"dq": dq, "dk": dk, "dq_w": dq_w, "dk_w": dk_w}


def rglru_local_attention(q, k, v, o, window, sinks=0, lens=None, scale=0.0, lse=None, stream=None):
    """q [B,T,Hq,dh], k, v [B,T,Hkv,dh], o as q and contiguous, bf16; lens int32 [B]; lse f32
    [B,Hq,T]."""
    _call("rglru_local_attention", _ext.local_attention, q, stream, q, k, v, lens, o, lse,
          window, sinks, scale)


def local_attention(q, k, v, window, sinks=0, lens=None, scale=0.0, want_lse=False, stream=None):
    """Returns o [B,T,Hq,dh] (bf16), or (o, lse) with lse f32 [B,Hq,T], which the backward needs."""
    if stream is not None:
        return _on(stream, q, lambda: local_attention(q, k, v, window, sinks, lens, scale, want_lse))
    o, lse = _ext.empty_as(q), None
    if want_lse:
        B, T, Hq, _ = q.shape
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    rglru_local_attention(q, k, v, o, window, sinks, lens, scale, lse)
    return (o, lse) if want_lse else o


def rglru_local_attention_backward_workspace_size(B, T, Hq, Hkv, dh, window, sinks=0) -> int:
    return int(_lib.rglru_local_attention_backward_workspace_size(
        B, T, Hq, Hkv, dh, _int32(window), _int32(sinks)))


def rglru_local_attention_backward(q, k, v, o, lse, do, dq, dk, dv, window, sinks=0, lens=None,
                                   scale=0.0, workspace=None, stream=None):
    """o, do as q and contiguous; dq as q, dk and dv as k (slices of a packed gradient are fine)."""
    _call("rglru_local_attention_backward", _ext.local_attention_backward, q, stream, q, k, v,
          lens, o, lse, do, dq, dk, dv, window, sinks, scale, workspace)


def local_attention_backward(q, k, v, o, lse, do, window, sinks=0, lens=None, scale=0.0, dq=None,
                             dk=None, dv=None, workspace=None, stream=None):
    """Gradients through local_attention(.., want_lse=True). Returns a dict with dq, dk, dv (bf16;
    new contiguous tensors unless given)."""
    if stream is not None:
        return _on(stream, q, lambda: local_attention_backward(q, k, v, o, lse, do, window, sinks, lens, scale,
                                                               dq, dk, dv, workspace))

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=q.device)

    dq = empty(q.shape, q.dtype) if dq is None else dq
    dk = empty(k.shape, k.dtype) if dk is None else dk
    dv = empty(v.shape, v.dtype) if dv is None else dv
    if workspace is None and q.dim() == 4 and k.dim() == 4:
        n = rglru_local_attention_backward_workspace_size(*q.shape[:3], k.shape[2], q.shape[3],
                                                          window, sinks)
        workspace = empty((n,), torch.uint8)
    rglru_local_attention_backward(q, k, v, o, lse, do, dq, dk, dv, window, sinks, lens, scale,
                                   workspace)
    return {"dq": dq, "dk": dk, "dv": dv}


@functools.lru_cache(maxsize=256)
def _paged_bytes(N, Hq, Hkv, dh, page_size, max_pages, window, sinks, dtype) -> int:
    return int(_lib.rglru_paged_attention_workspace_size(N, Hq, Hkv, dh, page_size, max_pages, window, sinks,
                                                         _dt(dtype)))


def rglru_paged_attention_workspace_size(N, Hq, Hkv, dh, page_size, max_pages, window, sinks,
                                         dtype) -> int:
    # (plain integers: a size must not be remembered for a tensor, whose value may change)
    return _paged_bytes(N, Hq, Hkv, dh, page_size, max_pages, _int32(window), _int32(sinks), dtype)


def rglru_paged_attention(q, k_pages, v_pages, block_table, lens, o, window, sinks=0, scale=0.0,
                          workspace=None, stream=None):
    """q [N,Hq,dh], k_pages, v_pages [pages,page,Hkv,dh] of one type (bf16 or f32); block_table
    int32 [N,max_pages], lens int32 [N]; o as q and contiguous."""
    _call("rglru_paged_attention", _ext.paged_attention, q, stream, q, k_pages, v_pages,
          block_table, lens, o, window, sinks, scale, workspace)


def paged_attention(q, k_pages, v_pages, block_table, lens, window, sinks=0, scale=0.0,
                    workspace=None, stream=None):
    """Returns o [N,Hq,dh] of q's type."""
    if stream is not None:
        return _on(stream, q, lambda: paged_attention(q, k_pages, v_pages, block_table, lens, window, sinks,
                                                      scale, workspace))
    o = _ext.empty_as(q)
    if workspace is None and q.dim() == 3 and k_pages.dim() == 4 and block_table.dim() == 2:
        N, Hq, dh = q.shape
        _, page, Hkv, _ = k_pages.shape
        n = rglru_paged_attention_workspace_size(N, Hq, Hkv, dh, page, block_table.shape[1], window,
                                                 sinks, q.dtype)
        if n:
            workspace = _ext.empty_bytes(q, n)
    rglru_paged_attention(q, k_pages, v_pages, block_table, lens, o, window, sinks, scale, workspace)
    return o


# ---- convenience wrappers (allocate outputs with torch, then call the entry points above) ----
def pre_buffer(x):
    """An empty pre-activation buffer in the layout rglru_gate_preacts writes."""
    B, T, D = x.shape
    if x.dtype == torch.bfloat16:
        return torch.empty((B, T, D), dtype=torch.int32, device=x.device)
    return torch.empty((B, T, D, 2), dtype=torch.float32, device=x.device)


def forward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0=None, plan="auto", chunk_len=0,
            workspace=None, stream=None):
    """Returns (y, h_T)."""
    if stream is not None:
        return _on(stream, x, lambda: forward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, plan, chunk_len,
                                              workspace))
    B, T, D = x.shape
    H = W_a.shape[0]
    y = torch.empty_like(x)
    h_T = torch.empty((B, D), dtype=torch.float32, device=x.device)
    if workspace is None:
        n = rglru_forward_workspace_size_planned(B, T, D, H, x.dtype, plan, chunk_len)
        if n == 0:
            raise RglruError(RGLRU_ERR_UNSUPPORTED if plan == "fused" else RGLRU_ERR_INVALID_ARG,
                             "rglru_forward_workspace_size_planned")
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    rglru_forward_planned(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, h_T, workspace, plan,
                          chunk_len)
    return y, h_T


def decode_step(x_t, conv_state, h, conv_w, W_a, b_a, W_x, b_x, Lambda, stream=None):
    """In place on conv_state and h; returns y_t."""
    if stream is not None:
        return _on(stream, x_t, lambda: decode_step(x_t, conv_state, h, conv_w, W_a, b_a, W_x, b_x, Lambda))
    y_t = torch.empty_like(x_t)
    rglru_decode_step(x_t, conv_state, h, y_t, conv_w, W_a, b_a, W_x, b_x, Lambda)
    return y_t


def backward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, dy, dh_T=None, want_dh0=True,
             workspace=None, stream=None):
    """Gradients through the forward. Returns a dict with dx (x's dtype) and fp32 dconv_w [4,D],
    dW_a, dW_x [H,Dh,Dh], db_a, db_x, dLam [D] and dh0 [B,D] (None unless want_dh0)."""
    if stream is not None:
        return _on(stream, x, lambda: backward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, dy, dh_T,
                                               want_dh0, workspace))
    B, T, D = x.shape
    H = W_a.shape[0]
    Dh = D // H
    dev = x.device
    f32 = torch.float32
    out = {"dx": torch.empty_like(x), "dconv_w": torch.empty((4, D), dtype=f32, device=dev),
           "dW_a": torch.empty((H, Dh, Dh), dtype=f32, device=dev),
           "db_a": torch.empty(D, dtype=f32, device=dev),
           "dW_x": torch.empty((H, Dh, Dh), dtype=f32, device=dev),
           "db_x": torch.empty(D, dtype=f32, device=dev),
           "dLam": torch.empty(D, dtype=f32, device=dev),
           "dh0": torch.empty((B, D), dtype=f32, device=dev) if want_dh0 else None}
    if workspace is None:
        workspace = torch.empty(rglru_backward_workspace_size(B, T, D, H, x.dtype),
                                dtype=torch.uint8, device=dev)
    rglru_backward(x, conv_w, W_a, b_a, W_x, b_x, Lambda, h0, y, dy, dh_T, out["dx"],
                   out["dconv_w"], out["dW_a"], out["db_a"], out["dW_x"], out["db_x"],
                   out["dLam"], out["dh0"], workspace)
    return out
