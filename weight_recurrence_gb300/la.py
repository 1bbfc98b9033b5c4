"""ctypes binding of liblinattn.so (argument marshalling only).

Every function here has the name of the C entry point it calls (see
``include/la.h``) and takes torch tensors for the device buffers; torch
provides device memory and the current CUDA stream, nothing else.  All work
runs in the library's kernels.  If the library is missing the first call
raises: there is no fallback.

Two builds of the library exist: liblinattn.so (the product) and
liblinattn_checked.so, the same kernels compiled with in-kernel bounds checks
that record LA_ERR_BOUNDS in the error word instead of making an access out
of range.  The environment variable LA_CHECKED=1 (read at the first load) or
select_library(checked=True) makes every call below go to the checked build.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "liblinattn.so")
LIB_CHECKED_PATH = os.path.join(_PKG, "lib", "liblinattn_checked.so")
BINDING_PATH = os.path.join(_PKG, "lib", "_la_torch.so")

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_BOUNDS = range(6)
LA_DTYPE_F32, LA_DTYPE_BF16 = 0, 1
LA_OP_NONCAUSAL, LA_OP_CAUSAL, LA_OP_DECODE, LA_OP_NONCAUSAL_BWD, LA_OP_CAUSAL_BWD = 0, 1, 2, 3, 4

EXPORTED = ("la_workspace_bytes", "la_forward_noncausal", "la_forward_causal", "la_decode_step",
            "la_get_last_error", "la_status_string", "la_version", "la_launch_count",
            "la_debug_inject_timeout", "la_forward_noncausal_noalloc", "la_backward_causal",
            "la_backward_noncausal", "la_forward_causal_varlen", "la_decode_steps",
            "la_feature_dim", "la_variant_workspace_bytes", "la_forward_causal_variant",
            "la_forward_noncausal_variant", "la_decode_step_variant", "la_checked_build",
            "la_debug_inject_bounds", "la_recurrence_workspace_bytes",
            "la_recurrence_forward", "la_recurrence_step",
            "la_recurrence_backward", "la_layernorm_forward", "la_layernorm_workspace_bytes",
            "la_layernorm_backward", "la_grad_workspace_bytes", "la_grad_norm", "la_grad_clip",
            "la_decay_forward", "la_decay_workspace_bytes", "la_decay_step", "la_decay_backward",
            "la_qk_rotate_forward", "la_qk_rotate_workspace_bytes", "la_qk_rotate_backward")

LA_FM = {"elu1": 0, "dpfp": 1, "poly2": 2}
LA_NORM = {"den": 0, "sum": 1, "none": 2}
LA_UPDATE = {"sum": 0, "delta": 1}
LA_GATE = {"decay": 0, "log": 1, "sigmoid": 2}
LA_PAIRS = {"half": 0, "adjacent": 1}


class LAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


class la_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("D", ctypes.c_int), ("M", ctypes.c_int), ("dtype", ctypes.c_int)]


class la_variant(ctypes.Structure):
    _fields_ = [("feature_map", ctypes.c_int), ("nu", ctypes.c_int), ("norm", ctypes.c_int),
                ("update", ctypes.c_int)]


class la_view(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong),
                ("sn", ctypes.c_longlong)]


class la_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_longlong)]


class la_tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_longlong),
                ("dtype", ctypes.c_int)]


class la_rotation(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("sa", ctypes.c_longlong), ("sb", ctypes.c_longlong),
                ("sn", ctypes.c_longlong), ("freq", ctypes.c_void_p), ("axes", ctypes.c_char_p), ("A", ctypes.c_int),
                ("P", ctypes.c_int), ("pairs", ctypes.c_int)]


class la_qk_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("D", ctypes.c_int), ("dtype", ctypes.c_int)]


def variant(fm: str = "elu1", nu: int = 1, norm: str = "den", update: str = "sum") -> la_variant:
    """la_variant from names: fm in {"elu1", "dpfp", "poly2"}, norm in {"den",
    "sum", "none"}, update in {"sum", "delta"}."""
    return la_variant(LA_FM[fm], int(nu), LA_NORM[norm], LA_UPDATE[update])


_lib = None
_loaded = {}


def select_library(checked: bool) -> ctypes.CDLL:
    """Routes the calls of this module to the checked build (True) or to the
    product build (False); returns the library now in use."""
    global _lib
    _lib = _load(LIB_CHECKED_PATH if checked else LIB_PATH)
    return _lib


def lib() -> ctypes.CDLL:
    """The library in use (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_CHECKED_PATH if os.environ.get("LA_CHECKED", "0") not in ("", "0") else LIB_PATH)
    return _lib


def _load(path: str) -> ctypes.CDLL:
    L = _loaded.get(path)
    if L is None:
        if not os.path.exists(path):
            flag = " --checked" if path == LIB_CHECKED_PATH else ""
            raise RuntimeError("%s is not built; run `python -m weight_recurrence_gb300.build%s`"
                               % (path, flag))
        L = ctypes.CDLL(path)
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.la_workspace_bytes.restype = sz
        L.la_workspace_bytes.argtypes = [i, la_shape, i]
        L.la_forward_noncausal.restype = i
        L.la_forward_noncausal.argtypes = [vp, vp, vp, vp, la_shape, vp, sz, vp]
        L.la_forward_causal.restype = i
        L.la_forward_causal.argtypes = [vp, vp, vp, vp, la_shape, i, vp, vp, vp, sz, vp]
        L.la_decode_step.restype = i
        L.la_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, la_shape, vp]
        L.la_get_last_error.restype = i
        L.la_get_last_error.argtypes = [vp]
        L.la_status_string.restype = ctypes.c_char_p
        L.la_status_string.argtypes = [i]
        L.la_version.restype = i
        L.la_launch_count.restype = ctypes.c_ulonglong
        L.la_forward_noncausal_noalloc.restype = i
        L.la_forward_noncausal_noalloc.argtypes = [vp, vp, vp, vp, la_shape, vp]
        L.la_debug_inject_timeout.restype = None
        L.la_debug_inject_timeout.argtypes = [i, i]
        L.la_backward_causal.restype = i
        L.la_backward_causal.argtypes = [vp, vp, vp, vp, vp, vp, vp, la_shape, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.la_forward_causal_varlen.restype = i
        L.la_forward_causal_varlen.argtypes = [vp, vp, vp, vp, vp, la_shape, vp, vp, vp, sz, vp]
        L.la_decode_steps.restype = i
        L.la_decode_steps.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, la_shape, vp]
        L.la_backward_noncausal.restype = i
        L.la_backward_noncausal.argtypes = [vp, vp, vp, vp, vp, vp, vp, la_shape, vp, sz, vp]
        L.la_feature_dim.restype = i
        L.la_feature_dim.argtypes = [la_variant, i]
        L.la_variant_workspace_bytes.restype = sz
        L.la_variant_workspace_bytes.argtypes = [i, la_shape, la_variant]
        L.la_forward_causal_variant.restype = i
        L.la_forward_causal_variant.argtypes = [vp, vp, vp, vp, vp, la_shape, la_variant, vp, vp, vp]
        L.la_forward_noncausal_variant.restype = i
        L.la_forward_noncausal_variant.argtypes = [vp, vp, vp, vp, la_shape, la_variant, vp, sz, vp]
        L.la_decode_step_variant.restype = i
        L.la_decode_step_variant.argtypes = [vp, vp, vp, vp, vp, vp, vp, la_shape, la_variant, vp]
        L.la_checked_build.restype = i
        L.la_checked_build.argtypes = []
        L.la_debug_inject_bounds.restype = None
        L.la_debug_inject_bounds.argtypes = [i]
        ll, f = ctypes.c_longlong, ctypes.c_float
        L.la_recurrence_forward.restype = i
        L.la_recurrence_forward.argtypes = [la_view, la_view, la_view, vp, la_shape, i, vp, vp, vp, sz, vp]
        L.la_recurrence_workspace_bytes.restype = sz
        L.la_recurrence_workspace_bytes.argtypes = [la_shape]
        L.la_recurrence_step.restype = i
        L.la_recurrence_step.argtypes = [la_view, la_view, la_view, la_shape, i, vp, vp]
        L.la_recurrence_backward.restype = i
        L.la_recurrence_backward.argtypes = [la_view] * 6 + [vp, la_shape, i, vp, vp, vp, vp, sz, vp]
        L.la_layernorm_forward.restype = i
        L.la_layernorm_forward.argtypes = [la_rows] * 4 + [vp, vp, vp, vp, ll, i, i, f, vp]
        L.la_layernorm_workspace_bytes.restype = sz
        L.la_layernorm_workspace_bytes.argtypes = [ll, i, i]
        L.la_layernorm_backward.restype = i
        L.la_layernorm_backward.argtypes = [la_rows] * 4 + [vp, vp, vp, vp, vp, ll, i, i, vp, sz, vp]
        L.la_grad_workspace_bytes.restype = sz
        L.la_grad_workspace_bytes.argtypes = [i]
        L.la_grad_norm.restype = i
        L.la_grad_norm.argtypes = [vp, i, vp, vp, sz, vp]
        L.la_grad_clip.restype = i
        L.la_grad_clip.argtypes = [vp, i, f, vp, vp, sz, vp]
        L.la_decay_forward.restype = i
        L.la_decay_forward.argtypes = [la_view] * 4 + [vp, vp, la_shape, f, vp, vp, vp, sz, vp]
        L.la_decay_workspace_bytes.restype = sz
        L.la_decay_workspace_bytes.argtypes = [la_shape, i]
        L.la_decay_step.restype = i
        L.la_decay_step.argtypes = [la_view] * 4 + [vp, la_shape, f, vp, vp]
        L.la_decay_backward.restype = i
        L.la_decay_backward.argtypes = [la_view] * 7 + [vp, vp, la_shape, f, vp, vp, vp, vp, sz, vp]
        L.la_qk_rotate_forward.restype = i
        L.la_qk_rotate_forward.argtypes = [la_view] * 4 + [vp, vp, la_rotation, la_qk_shape, i, f, vp]
        L.la_qk_rotate_workspace_bytes.restype = sz
        L.la_qk_rotate_workspace_bytes.argtypes = [la_qk_shape]
        L.la_qk_rotate_backward.restype = i
        L.la_qk_rotate_backward.argtypes = [la_view] * 6 + [vp, vp, la_rotation, la_qk_shape, i, f, vp, vp, vp, sz, vp]
        _loaded[path] = L
    return L


def status_string(st: int) -> str:
    return lib().la_status_string(int(st)).decode()


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return LA_DTYPE_F32
    if t == torch.bfloat16:
        return LA_DTYPE_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _stream(stream, device):
    return ctypes.c_void_p(_stream_ptr(stream, device))


def _check(st: int, where: str):
    if st != LA_OK:
        raise LAError(st, where)


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def shape_of(q: torch.Tensor, v: torch.Tensor) -> la_shape:
    B, H, N, D = q.shape
    return la_shape(B, H, N, D, v.shape[-1], _dtype_code(q.dtype))


_SIZE_MAX = ctypes.c_size_t(-1).value
_ws_bytes_cache = {}


def la_workspace_bytes(op: int, shape: la_shape, chunk: int = 0) -> int:
    key = (int(op), shape.B, shape.H, shape.N, shape.D, shape.M, shape.dtype, int(chunk))
    n = _ws_bytes_cache.get(key)
    if n is None:
        n = lib().la_workspace_bytes(int(op), shape, int(chunk))
        if n == _SIZE_MAX:
            raise LAError(LA_ERR_INVALID_ARG, "la_workspace_bytes")
        _ws_bytes_cache[key] = n = int(n)
    return n


_ws_cache = {}


def _workspace(nbytes: int, device, stream_ptr: int) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    key = (device.index, stream_ptr)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def la_forward_noncausal(q, k, v, out=None, stream=None):
    """V' = phi(Q)(phi(K)^T V) / phi(Q) sum phi(K) for q, k [B,H,N,D], v [B,H,N,M]."""
    _contig(q, k, v)
    s = shape_of(q, v)
    if out is None:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    need = la_workspace_bytes(LA_OP_NONCAUSAL, s, 0)
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(need, q.device, sp)
    st = lib().la_forward_noncausal(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, _ptr(ws), need, ctypes.c_void_p(sp))
    _check(st, "la_forward_noncausal")
    return out


def la_forward_noncausal_noalloc(q, k, v, out=None, stream=None):
    """As la_forward_noncausal, but the library uses its own fixed 8 MiB device
    scratch array instead of a workspace (for callers that cannot allocate;
    overlapping calls race on that array)."""
    _contig(q, k, v)
    s = shape_of(q, v)
    if out is None:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    st = lib().la_forward_noncausal_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, _stream(stream, q.device))
    _check(st, "la_forward_noncausal_noalloc")
    return out


def la_forward_causal(q, k, v, out=None, chunk=0, S=None, z=None, want_out=True, stream=None):
    """Causal form (sums over j <= i).  S [B,H,D,M] / z [B,H,D] fp32, if given,
    hold the carried-in state and receive the state after the last token."""
    _contig(q, k, v, S, z)
    s = shape_of(q, v)
    if out is None and want_out:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    need = la_workspace_bytes(LA_OP_CAUSAL, s, chunk)
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(need, q.device, sp)
    st = lib().la_forward_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, int(chunk), _ptr(S), _ptr(z),
                                 _ptr(ws), need, ctypes.c_void_p(sp))
    _check(st, "la_forward_causal")
    return out


def la_decode_step(q, k, v, S, z, y=None, stream=None):
    """One recurrent step for q, k [B,H,D], v [B,H,M]; S, z fp32 updated in place."""
    _contig(q, k, v, S, z)
    B, H, D = q.shape
    M = v.shape[-1]
    if y is None:
        y = torch.empty((B, H, M), dtype=q.dtype, device=q.device)
    _contig(y)
    s = la_shape(B, H, 1, D, M, _dtype_code(q.dtype))
    st = lib().la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(S), _ptr(z), s,
                              _stream(stream, q.device))
    _check(st, "la_decode_step")
    return y


def la_forward_causal_varlen(q, k, v, lens, out=None, S=None, z=None, want_out=True, stream=None):
    """Causal form for a batch of sequences of lengths lens [B] (int32, on the
    device); rows past a sequence's length are ignored (their output rows are
    unspecified).  S, z as in la_forward_causal, per sequence."""
    _contig(q, k, v, S, z, lens)
    if lens.dtype != torch.int32:
        raise ValueError("lens must be int32")
    s = shape_of(q, v)
    if out is None and want_out:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    need = la_workspace_bytes(LA_OP_CAUSAL, s, 0)
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(need, q.device, sp)
    st = lib().la_forward_causal_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lens), s, _ptr(S), _ptr(z),
                                        _ptr(ws), need, ctypes.c_void_p(sp))
    _check(st, "la_forward_causal_varlen")
    return out


def la_decode_steps(q, k, v, S, z, y=None, steps=None, stream=None):
    """T recurrent steps in one launch: q, k [T,B,H,D], v [T,B,H,M]; S, z fp32
    updated in place; steps: optional int32 [B] per-sequence step counts."""
    _contig(q, k, v, S, z, steps)
    T, B, H, D = q.shape
    M = v.shape[-1]
    if y is None:
        y = torch.empty((T, B, H, M), dtype=q.dtype, device=q.device)
    _contig(y)
    if steps is not None and steps.dtype != torch.int32:
        raise ValueError("steps must be int32")
    s = la_shape(B, H, 1, D, M, _dtype_code(q.dtype))
    st = lib().la_decode_steps(_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(S), _ptr(z), _ptr(steps), int(T), s,
                               _stream(stream, q.device))
    _check(st, "la_decode_steps")
    return y


def la_backward_causal(q, k, v, dout, dq=None, dk=None, dv=None, S0=None, z0=None, dSN=None, dzN=None,
                       dS0=None, dz0=None, stream=None):
    """Gradients dq, dk, dv of the causal form given dout = dL/dV'.  S0/z0: the
    state the forward started from; dSN/dzN: gradient reaching its final
    state; dS0/dz0 (fp32, written): gradient of the starting state."""
    _contig(q, k, v, dout, S0, z0, dSN, dzN, dS0, dz0)
    s = shape_of(q, v)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _contig(dq, dk, dv)
    need = la_workspace_bytes(LA_OP_CAUSAL_BWD, s, 0)
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(need, q.device, sp)
    st = lib().la_backward_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), s,
                                  _ptr(S0), _ptr(z0), _ptr(dSN), _ptr(dzN), _ptr(dS0), _ptr(dz0),
                                  _ptr(ws), need, ctypes.c_void_p(sp))
    _check(st, "la_backward_causal")
    return dq, dk, dv


def la_backward_noncausal(q, k, v, dout, dq=None, dk=None, dv=None, stream=None):
    """Gradients dq, dk, dv of the non-causal form given dout = dL/dV'."""
    _contig(q, k, v, dout)
    s = shape_of(q, v)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _contig(dq, dk, dv)
    need = la_workspace_bytes(LA_OP_NONCAUSAL_BWD, s, 0)
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(need, q.device, sp)
    st = lib().la_backward_noncausal(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), s,
                                     _ptr(ws), need, ctypes.c_void_p(sp))
    _check(st, "la_backward_noncausal")
    return dq, dk, dv


def la_feature_dim(var: la_variant, D: int) -> int:
    """Width F of phi(x) for x in R^D under the variant (0 if invalid)."""
    return int(lib().la_feature_dim(var, int(D)))


def la_forward_causal_variant(q, k, v, var: la_variant, beta=None, out=None, S=None, z=None, want_out=True,
                              stream=None):
    """Causal form of a variant: q, k [B,H,N,D], v [B,H,N,M], beta [B,H,N]
    (delta rule).  S [B,H,F,M] (and z [B,H,F] with the denominator) fp32, if
    given, hold the starting state and receive the final one."""
    _contig(q, k, v, beta, S, z)
    s = shape_of(q, v)
    if out is None and want_out:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    st = lib().la_forward_causal_variant(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(out), s, var, _ptr(S),
                                         _ptr(z), _stream(stream, q.device))
    _check(st, "la_forward_causal_variant")
    return out


def la_forward_noncausal_variant(q, k, v, var: la_variant, out=None, stream=None):
    """Non-causal form of a variant (sum update)."""
    _contig(q, k, v)
    s = shape_of(q, v)
    if out is None:
        out = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    _contig(out)
    need = lib().la_variant_workspace_bytes(LA_OP_NONCAUSAL, s, var)
    if need == _SIZE_MAX:
        raise LAError(LA_ERR_UNSUPPORTED, "la_variant_workspace_bytes")
    sp = _stream_ptr(stream, q.device)
    ws = _workspace(int(need), q.device, sp)
    st = lib().la_forward_noncausal_variant(_ptr(q), _ptr(k), _ptr(v), _ptr(out), s, var, _ptr(ws), int(need),
                                            ctypes.c_void_p(sp))
    _check(st, "la_forward_noncausal_variant")
    return out


def la_decode_step_variant(q, k, v, S, var: la_variant, z=None, beta=None, y=None, stream=None):
    """One recurrent step of a variant: q, k [B,H,D], v [B,H,M], beta [B,H];
    S [B,H,F,M] (and z [B,H,F] with the denominator) updated in place."""
    _contig(q, k, v, S, z, beta)
    B, H, D = q.shape
    M = v.shape[-1]
    if y is None:
        y = torch.empty((B, H, M), dtype=q.dtype, device=q.device)
    _contig(y)
    s = la_shape(B, H, 1, D, M, _dtype_code(q.dtype))
    st = lib().la_decode_step_variant(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(y), _ptr(S), _ptr(z), s, var,
                                      _stream(stream, q.device))
    _check(st, "la_decode_step_variant")
    return y


# ------------------------------------------- the layer around the attention
# Their binding is compiled (csrc/la_torch.cpp): it checks shapes, types and
# devices, takes views, allocates what a call returns or needs as workspace on
# the stream that it launches on, and calls the library in use.  Raises
# ValueError or TypeError for arguments it refuses, LAError for what the library
# answers.

_binding = None
_binding_for = None


def _bound():
    """The compiled binding, calling the library in use."""
    global _binding, _binding_for
    L = lib()
    if _binding_for is not L:
        if _binding is None:
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError("%s is not built; run `python -m weight_recurrence_gb300.build`" % BINDING_PATH)
            loader = importlib.machinery.ExtensionFileLoader("_la_torch", BINDING_PATH)
            spec = importlib.util.spec_from_file_location("_la_torch", BINDING_PATH, loader=loader)
            _binding = importlib.util.module_from_spec(spec)
            loader.exec_module(_binding)
        _binding.use(L._name)
        _binding_for = L
    return _binding


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _gate_code(gate: str) -> int:
    code = LA_GATE.get(gate)
    if code is None:
        raise ValueError("gate must be one of %s" % ", ".join(LA_GATE))
    return code


def la_recurrence_forward(x, g, gate="sigmoid", out=None, h0=None, hN=None, lens=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t of every channel, out_t = h_t.

    x, g: [B,N,D] or [B,H,N,D], any strides but the channels'.  gate: "decay"
    (a = g, u = x), "log" (a = e^g, u = x) or "sigmoid" (a = sigmoid(g),
    u = (1 - a) x).  h0, hN: fp32 states [B,D] or [B,H,D], read before the
    first token and written after the last; hN may be h0.  lens: int32 [B];
    rows past a length are 0.  Returns out."""
    st, out = _bound().recurrence_forward(x, g, _gate_code(gate), out, h0, hN, lens, _handle(stream))
    _check(st, "la_recurrence_forward")
    return out


def la_recurrence_step(x, g, h, gate="sigmoid", y=None, stream=None):
    """One token of the recurrence: x, g [B,D] or [B,H,D]; h the fp32 state of
    the same shape, updated in place.  Returns y = h in x's type."""
    st, y = _bound().recurrence_step(x, g, h, _gate_code(gate), y, _handle(stream))
    _check(st, "la_recurrence_step")
    return y


def la_recurrence_backward(x, g, out, dout, gate="sigmoid", h0=None, dhN=None, dh0=None, lens=None, dx=None, dg=None,
                           stream=None):
    """Gradients (dx, dg) of la_recurrence_forward given its out and dout =
    dL/dout.  h0, lens: as given to the forward; dhN: gradient of its hN; dh0
    (fp32, written): gradient of h0, may be dhN.  x is read by the sigmoid
    gate only and may be None for the others."""
    st, dx, dg = _bound().recurrence_backward(x, g, out, dout, _gate_code(gate), h0, dhN, dh0, lens, dx, dg,
                                              _handle(stream))
    _check(st, "la_recurrence_backward")
    return dx, dg


def la_layernorm_forward(x, w=None, b=None, eps=1e-5, res=None, y=None, sum=None, mean=None, rstd=None, stats=True,
                         stream=None):
    """Layer norm of the rows of x [..., C], with the residual sum s = x + res
    in front when res is given.  w, b: fp32 [C] or None.  Returns (y, s, mean,
    rstd): s is x itself without res; mean and rstd (fp32, for the backward)
    are None with stats=False.  sum: where s goes (may be x or res)."""
    st, y, s, mean, rstd = _bound().layernorm_forward(x, w, b, eps, res, y, sum, mean, rstd, stats, _handle(stream))
    _check(st, "la_layernorm_forward")
    return y, s, mean, rstd


def la_layernorm_backward(dy, s, w, mean, rstd, dsum=None, ds=None, dw=None, db=None, stream=None):
    """Gradients (ds, dw, db) of la_layernorm_forward given dy = dL/dy, the s,
    mean and rstd it returned and, where s went on as the residual stream,
    dsum = dL/ds.  ds is the gradient of x and of res; w may be None (1)."""
    st, ds, dw, db = _bound().layernorm_backward(dy, s, w, mean, rstd, dsum, ds, dw, db, _handle(stream))
    _check(st, "la_layernorm_backward")
    return ds, dw, db


def la_grad_norm(grads, norm=None, stream=None):
    """Global norm sqrt(sum of all squares) over a list of contiguous tensors,
    an fp32 scalar on the device."""
    st, norm = _bound().grad(grads, None, None, norm, _handle(stream))
    _check(st, "la_grad_norm")
    return norm


def la_grad_clip(grads, max_norm, out=None, norm=None, stream=None):
    """Scales every tensor of a list by min(1, max_norm / (norm + 1e-6)) with
    the global norm, in place or into the tensors of out; returns the norm (an
    fp32 scalar on the device).  No tensor may be listed twice, nor be the out of
    another (LAError)."""
    st, norm = _bound().grad(grads, float(max_norm), out, norm, _handle(stream))
    _check(st, "la_grad_clip")
    return norm


def la_decay_forward(q, k, v, log_decay, scale=1.0, S0=None, SN=None, lens=None, out=None, want_out=True, stream=None):
    """Linear attention with a decay for each head: S_i = e^g S_{i-1} + k_i v_i^T,
    out_i = scale q_i^T S_i, g = log_decay[h].

    q, k: [B,H,N,D], v: [B,H,N,M], any strides but the channels'; log_decay: fp32
    [H], at most 0 for states that do not grow, at most 1/2 for ones that do.  S0, SN: fp32 [B,H,D,M], the
    state before the first token and after the last; SN may be S0.  lens: int32
    [B]; rows past a length are 0.  want_out=False: the state alone (q may be
    None).  Returns out."""
    st, out = _bound().decay_forward(q, k, v, log_decay, scale, S0, SN, lens, out, bool(want_out), _handle(stream))
    _check(st, "la_decay_forward")
    return out


def la_decay_step(q, k, v, S, log_decay, scale=1.0, y=None, stream=None):
    """One token: q, k [B,H,D], v [B,H,M]; S the fp32 state [B,H,D,M], updated in
    place.  Returns y = scale q^T S in v's type."""
    st, y = _bound().decay_step(q, k, v, S, log_decay, scale, y, _handle(stream))
    _check(st, "la_decay_step")
    return y


def la_decay_backward(q, k, v, dout, log_decay, scale=1.0, S0=None, dSN=None, dS0=None, lens=None, dq=None, dk=None,
                      dv=None, stream=None):
    """Gradients (dq, dk, dv) of la_decay_forward given dout = dL/dout.  S0, lens:
    as given to the forward; dSN: gradient of its SN; dS0 (fp32, written):
    gradient of S0.  log_decay gets none."""
    st, dq, dk, dv = _bound().decay_backward(q, k, v, dout, log_decay, scale, S0, dSN, dS0, lens, dq, dk, dv,
                                             _handle(stream))
    _check(st, "la_decay_backward")
    return dq, dk, dv


def _pairs_code(pairs: str) -> int:
    code = LA_PAIRS.get(pairs)
    if code is None:
        raise ValueError("pairs must be one of %s" % ", ".join(LA_PAIRS))
    return code


def _axes_bytes(axes):
    # (bytes() of an integer or of an array would be something else)
    return axes if axes is None else bytes(axes if isinstance(axes, (bytes, tuple, list)) else [int(i) for i in axes])


def la_qk_rotate_forward(q, k, pos, freq, wq=None, wk=None, eps=1e-6, norm=True, pairs="half", axes=None, qo=None,
                         ko=None, stream=None):
    """RMS norm of every head of q [B,Hq,N,D] and k [B,Hk,N,D] (or None) and the
    rotation of its first 2 P channels by the angles position * freq, P =
    len(freq), in one pass.

    pos: int32 [N], [B,N] or [A,B,N] (A axes, as time, height and width); freq:
    fp32 [P]; axes: the axis of each of the P pairs (None: all on the first).
    pairs: "half" (channels i and i + P) or "adjacent" (2i and 2i + 1).  wq, wk:
    fp32 [D] or None (1); norm=False: the rotation alone.  qo may be q, ko may be
    k.  Returns (qo, ko)."""
    st, qo, ko = _bound().qk_rotate_forward(q, k, pos, freq, wq, wk, eps, bool(norm), _pairs_code(pairs),
                                            _axes_bytes(axes), qo, ko, _handle(stream))
    _check(st, "la_qk_rotate_forward")
    return qo, ko


def la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq=None, wk=None, eps=1e-6, norm=True, pairs="half", axes=None,
                          dq=None, dk=None, dwq=None, dwk=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of la_qk_rotate_forward given dqo, dko and its
    own inputs; dwq, dwk (fp32 [D]) are None with norm=False, dk and dwk without
    keys.  dq may be dqo, dk may be dko."""
    st, dq, dk, dwq, dwk = _bound().qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk, eps, bool(norm),
                                                       _pairs_code(pairs), _axes_bytes(axes), dq, dk, dwq, dwk,
                                                       _handle(stream))
    _check(st, "la_qk_rotate_backward")
    return dq, dk, dwq, dwk


def la_get_last_error(stream=None, device=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    dev = device if device is not None else torch.cuda.current_device()
    return int(lib().la_get_last_error(_stream(stream, dev)))


def la_debug_inject_timeout(enable: bool, limit_us: int = 1000):
    lib().la_debug_inject_timeout(1 if enable else 0, int(limit_us))


def la_checked_build() -> bool:
    """True when the library in use is the bounds-checked build."""
    return bool(lib().la_checked_build())


def la_debug_inject_bounds(enable: bool):
    """Checked build only (a no-op otherwise): while enabled, the kernels that
    read a carried-in state or a workspace slot offset that index past its
    buffer, so that their check records LA_ERR_BOUNDS and skips the access."""
    lib().la_debug_inject_bounds(1 if enable else 0)


def la_version() -> int:
    return int(lib().la_version())


def la_launch_count() -> int:
    """Kernels launched through the library by this process so far."""
    return int(lib().la_launch_count())
