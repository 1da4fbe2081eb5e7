"""Gated DeltaNet-2 operator, and the other operators of its hybrid block (windowed
attention with sinks, gated linear recurrence, block norm), on B200: Python binding
of libgdn2.so.

The binding only marshals torch tensors (device memory) and the current CUDA
stream into the C ABI declared in ``include/gdn2.h``; every step of the
operator runs in the library's CUDA kernels.  There is no CPU fallback: if the
native library is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIBRARY_PATH = _PKG / "libgdn2.so"

GDN2_OK = 0
GDN2_ERR_NULL = 1
GDN2_ERR_SHAPE = 2
GDN2_ERR_DTYPE = 3
GDN2_ERR_ALIGN = 4
GDN2_ERR_UNSUPPORTED = 5
GDN2_ERR_CUDA = 6
GDN2_ERR_DEVICE_TIMEOUT = 7
GDN2_ERR_RANGE = 8
GDN2_ERR_SCRATCH_LIMIT = 9

GDN2_F32 = 0
GDN2_BF16 = 1

# gdn2_gate_layout bits: which gates hold one value per (token, head)
GDN2_GATES_PER_CHANNEL = 0
GDN2_ERASE_SCALAR = 1
GDN2_WRITE_SCALAR = 2
GDN2_DECAY_SCALAR = 4

# tokens between the checkpoints gdn2_scan_fwd leaves for gdn2_scan_bwd
GDN2_SCAN_BLOCK = 16

# Every symbol include/gdn2.h declares.
EXPORTED = ("gdn2_fwd_chunked", "gdn2_fwd_chunked_gates", "gdn2_fwd_chunked_noalloc",
            "gdn2_layer_fwd", "gdn2_bwd_chunked", "gdn2_decode_step", "gdn2_decode_tokens",
            "gdn2_swa_fwd", "gdn2_swa_bwd", "gdn2_swa_decode", "gdn2_scan_fwd", "gdn2_scan_bwd", "gdn2_scan_step",
            "gdn2_block_norm_fwd", "gdn2_block_norm_bwd", "gdn2_check_device_error", "gdn2_selftest_bounded_wait", "gdn2_fwd_chunked_launches", "gdn2_status_string")

_lib = None


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load libgdn2.so (built in-tree by ``gated_delta_rule_118_b200.build``)."""
    global _lib
    if _lib is None:
        if not LIBRARY_PATH.exists():
            raise RuntimeError(f"native library {LIBRARY_PATH} is missing; run "
                               "`python -m gated_delta_rule_118_b200.build` (there is no fallback)")
        L = ctypes.CDLL(str(LIBRARY_PATH))
        vp, fp, ci = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.gdn2_fwd_chunked.argtypes = [vp] * 5 + [fp, fp, vp, fp] + [ci] * 6 + [vp]
        L.gdn2_fwd_chunked.restype = ci
        L.gdn2_fwd_chunked_gates.argtypes = [vp] * 5 + [fp, fp, vp, fp] + [ci] * 6 + [ctypes.c_uint, vp]
        L.gdn2_fwd_chunked_gates.restype = ci
        L.gdn2_decode_tokens.argtypes = [vp] * 5 + [fp, fp, vp] + [ci] * 6 + [ctypes.c_uint, vp]
        L.gdn2_decode_tokens.restype = ci
        L.gdn2_layer_fwd.argtypes = [vp] * 5 + [fp, vp, fp, ctypes.c_float, fp, vp, fp] + [ci] * 6 + [vp]
        L.gdn2_layer_fwd.restype = ci
        L.gdn2_bwd_chunked.argtypes = [vp] * 5 + [fp, fp, vp, fp] + [fp] * 7 + [ci] * 6 + [vp]
        L.gdn2_bwd_chunked.restype = ci
        L.gdn2_fwd_chunked_noalloc.argtypes = [vp] * 5 + [fp, fp, vp, fp] + [ci] * 6 + [vp]
        L.gdn2_fwd_chunked_noalloc.restype = ci
        L.gdn2_decode_step.argtypes = [vp] * 5 + [fp, fp, vp] + [ci] * 5 + [vp]
        L.gdn2_decode_step.restype = ci
        cl, cf = ctypes.c_longlong, ctypes.c_float
        L.gdn2_swa_fwd.argtypes = [vp] * 6 + [ci] * 8 + [cf, vp, ci, vp]
        L.gdn2_swa_bwd.argtypes = [vp] * 10 + [ci] * 8 + [cf, vp, ci, vp]
        L.gdn2_swa_decode.argtypes = [vp] * 7 + [ci] * 7 + [cf, vp, ci, vp]
        L.gdn2_scan_fwd.argtypes = [vp] * 7 + [ci] * 4 + [vp]
        L.gdn2_scan_bwd.argtypes = [vp] * 10 + [ci] * 4 + [vp]
        L.gdn2_scan_step.argtypes = [vp] * 5 + [ci] * 3 + [vp]
        L.gdn2_block_norm_fwd.argtypes = [vp] * 6 + [cf] + [vp] * 2 + [cl, ci, ci, vp]
        L.gdn2_block_norm_bwd.argtypes = [vp] * 6 + [cf] + [vp] * 8 + [cl, ci, ci, vp]
        for fn in (L.gdn2_swa_fwd, L.gdn2_swa_bwd, L.gdn2_swa_decode, L.gdn2_scan_fwd, L.gdn2_scan_bwd,
                   L.gdn2_scan_step, L.gdn2_block_norm_fwd, L.gdn2_block_norm_bwd):
            fn.restype = ci
        L.gdn2_check_device_error.argtypes = [vp]
        L.gdn2_check_device_error.restype = ci
        L.gdn2_selftest_bounded_wait.argtypes = [vp]
        L.gdn2_selftest_bounded_wait.restype = ci
        L.gdn2_fwd_chunked_launches.argtypes = [ci] * 6
        L.gdn2_fwd_chunked_launches.restype = ci
        L.gdn2_status_string.argtypes = [ci]
        L.gdn2_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdn2_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN2_F32
    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _gate_layout(q, b, w, log_alpha):
    """gdn2_gate_layout bits from the shapes: a gate of shape q.shape[:-1] is per (token, head)."""
    tok = tuple(q.shape[:-1])
    return ((GDN2_ERASE_SCALAR if tuple(b.shape) == tok else 0)
            | (GDN2_WRITE_SCALAR if tuple(w.shape) == tok else 0)
            | (GDN2_DECAY_SCALAR if tuple(log_alpha.shape) == tok else 0))


def gdn2_fwd_chunked(q, k, v, b, w, log_alpha, S0=None, o=None, S_T=None, *,
                     stream=None, want_state=True, check=True):
    """Chunked forward.  Tensors are CUDA, contiguous, [B,T,H,d]; returns (o, S_T).

    ``o`` and ``S_T`` are allocated with torch when not given (S_T only when
    ``want_state``).  b, w or log_alpha of shape [B,T,H] (one value per token and
    head) select the matching gate layout (gdn2_fwd_chunked_gates).  Raises
    Gdn2Error on a non-OK status.
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("b", b), ("w", w), ("log_alpha", log_alpha),
                    ("o", o), ("S0", S0), ("S_T", S_T)):
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if log_alpha.dtype != torch.float32 or (S0 is not None and S0.dtype != torch.float32):
        raise TypeError("log_alpha and S0 must be float32")
    layout = _gate_layout(q, b, w, log_alpha)
    if layout:
        st = lib().gdn2_fwd_chunked_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(log_alpha),
                                          _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, _dtype_code(q),
                                          layout, _stream(stream))
    else:
        st = lib().gdn2_fwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(log_alpha),
                                    _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, _dtype_code(q),
                                    _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_fwd_chunked_gates" if layout else "gdn2_fwd_chunked")
    return o, S_T


def gdn2_fwd_chunked_noalloc(q, k, v, b, w, log_alpha, S0=None, o=None, S_T=None, *, stream=None,
                             check=True):
    """The chunked forward through the entry point that allocates no device memory.

    Pass ``o`` (and ``S_T`` when the final state is wanted) preallocated; the
    native call itself uses only its fixed scratch buffer.  Returns (o, S_T).
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        raise ValueError("gdn2_fwd_chunked_noalloc needs a preallocated output o")
    for name, t in (("q", q), ("k", k), ("v", v), ("b", b), ("w", w), ("log_alpha", log_alpha),
                    ("o", o), ("S0", S0), ("S_T", S_T)):
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    st = lib().gdn2_fwd_chunked_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w),
                                        _ptr(log_alpha), _ptr(S0), _ptr(o), _ptr(S_T),
                                        B, T, H, dk, dv, _dtype_code(q), _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_fwd_chunked_noalloc")
    return o, S_T


def gdn2_decode_step(q, k, v, b, w, log_alpha, S, o=None, *, stream=None, check=True):
    """One recurrent token: [B,H,d] inputs, S [B,H,dk,dv] fp32 updated in place; returns o."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    st = lib().gdn2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(log_alpha),
                                _ptr(S), _ptr(o), B, H, dk, dv, _dtype_code(q), _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_decode_step")
    return o


def gdn2_layer_fwd(q, k, v, b_logit, w_logit, decay_logit, g_logit, norm_weight, eps=1e-6, S0=None,
                   y=None, S_T=None, *, stream=None, want_state=True, check=True):
    """The operator with the layer's processing fused around it: L2-normalised q and
    k, sigmoid gates from logits, log_alpha = log sigmoid(decay_logit), and
    y = RMSNorm(o) * norm_weight * sigmoid(g_logit).  Tensors are CUDA, contiguous,
    [B,T,H,d] (norm_weight [dv] fp32, decay_logit fp32); returns (y, S_T)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if y is None:
        y = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("b_logit", b_logit), ("w_logit", w_logit),
                    ("decay_logit", decay_logit), ("g_logit", g_logit), ("norm_weight", norm_weight),
                    ("y", y), ("S0", S0), ("S_T", S_T)):
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if decay_logit.dtype != torch.float32 or norm_weight.dtype != torch.float32:
        raise TypeError("decay_logit and norm_weight must be float32")
    st = lib().gdn2_layer_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(b_logit), _ptr(w_logit), _ptr(decay_logit),
                              _ptr(g_logit), _ptr(norm_weight), ctypes.c_float(eps), _ptr(S0), _ptr(y),
                              _ptr(S_T), B, T, H, dk, dv, _dtype_code(q), _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_layer_fwd")
    return y, S_T


def gdn2_bwd_chunked(q, k, v, b, w, log_alpha, S0, dO, dS_T=None, *, stream=None, check=True,
                     want_dS0=True):
    """Backward of the chunked forward: gradients of sum(o * dO) + sum(S_T * dS_T).
    Inputs as for gdn2_fwd_chunked plus dO [B,T,H,dv] (input dtype) and dS_T
    [B,H,dk,dv] fp32 or None; returns a dict of fp32 tensors dq, dk, dv, db, dw,
    dlog_alpha and dS0 (None unless want_dS0)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {n: torch.empty((B, T, H, dk), **f32) for n in ("dq", "dk", "db", "dlog_alpha")}
    g.update({n: torch.empty((B, T, H, dv), **f32) for n in ("dv", "dw")})
    g["dS0"] = torch.empty((B, H, dk, dv), **f32) if want_dS0 else None
    for name, t in (("q", q), ("k", k), ("v", v), ("b", b), ("w", w), ("log_alpha", log_alpha),
                    ("S0", S0), ("dO", dO), ("dS_T", dS_T)):
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    st = lib().gdn2_bwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(log_alpha), _ptr(S0),
                                _ptr(dO), _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                                _ptr(g["db"]), _ptr(g["dw"]), _ptr(g["dlog_alpha"]), _ptr(g["dS0"]),
                                B, T, H, dk, dv, _dtype_code(q), _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_bwd_chunked")
    return g


def gdn2_decode_tokens(q, k, v, b, w, log_alpha, S, o=None, *, stream=None, check=True):
    """T recurrent tokens on a resident state: [B,T,H,d] inputs (b, w, log_alpha may be
    [B,T,H]: one value per token and head), S [B,H,dk,dv] fp32 updated in place;
    returns o [B,T,H,dv]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("b", b), ("w", w), ("log_alpha", log_alpha),
                    ("S", S), ("o", o)):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    st = lib().gdn2_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(log_alpha),
                                  _ptr(S), _ptr(o), B, T, H, dk, dv, _dtype_code(q),
                                  _gate_layout(q, b, w, log_alpha), _stream(stream))
    if check and st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_decode_tokens")
    return o


# ---------------------------------------------------------------- the hybrid block's other operators
_caller = None


_CALLS = ("gdn2_swa_fwd", "gdn2_swa_bwd", "gdn2_swa_decode", "gdn2_scan_fwd", "gdn2_scan_bwd", "gdn2_scan_step",
          "gdn2_block_norm_fwd", "gdn2_block_norm_bwd")


class _Ctypes:
    """The calls of module _call, through ctypes (2 to 4 microseconds more a call)."""

    def __init__(self, L):
        for name in _CALLS:
            setattr(self, name[len("gdn2_"):], self._of(getattr(L, name)))

    @staticmethod
    def _of(fn):
        sizes = [i for i, t in enumerate(fn.argtypes) if t is ctypes.c_int]

        def call(*args):
            if any(not -2 ** 31 <= args[i] < 2 ** 31 for i in sizes):  # (ctypes would cut it)
                raise OverflowError("a size does not fit 32 bits")
            return fn(*((ctypes.c_longlong * len(a))(*a) if isinstance(a, tuple) else a for a in args))
        return call


def _native():
    """What calls libgdn2.so for the functions below: the module built with it, else ctypes."""
    global _caller
    if _caller is None:
        L = lib()
        try:
            from . import _call as module
        except ImportError:
            module = _Ctypes(L)
        else:
            module.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _CALLS))
        _caller = module
    return _caller


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_cuda_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_CODE = {torch.float32: GDN2_F32, torch.bfloat16: GDN2_BF16}


def _here(first, stream):
    """The device of ``first`` if a call can be made as it stands (that device current, no stream given), else -1."""
    d = first.get_device()
    return d if d >= 0 and stream is None and d == _cuda_device() else -1


def _there(fn, stream, first, *args, **kw):
    """The call with ``first``'s device current, on ``stream`` if one is given (outputs are then
    allocated for that stream too), else on that device's current stream."""
    if not first.is_cuda:
        raise ValueError(f"{fn.__name__}: tensors must be CUDA tensors")
    if stream is not None:
        if stream.device != first.device:
            raise ValueError(f"{fn.__name__}: stream is on {stream.device}, tensors on {first.device}")
        with torch.cuda.stream(stream):
            return fn(first, *args, **kw)
    with torch.cuda.device(first.device):
        return fn(first, *args, **kw)


def _is(t, shape, dtype, dev):
    return t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _need(name, t, shape, dtype, dev, rows=False):
    """``t`` (None passes) is a dense tensor of this shape and type on device ``dev``; with ``rows``
    only its last axis has to be contiguous.  Raises otherwise."""
    if t is None or _is(t, shape, dtype, dev):
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if not rows:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")


def _code(t):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _p(t):
    return None if t is None else t.data_ptr()


def _done(st, check, where):
    if st != GDN2_OK and check:
        raise Gdn2Error(st, where)


def _strides(q, k, v):
    """The strides of all axes but the last; None if all three are dense."""
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        return None
    return (*q.stride()[:-1], *k.stride()[:-1], *v.stride()[:-1])


def _swa_sizes(q, k, v, lens, window, sinks, scale, dev):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,T,Hq,d], k and v [B,Tk,Hk,d]")
    B, T, Hq, d = q.shape
    _, Tk, Hk, _ = k.shape
    dt, code = q.dtype, _code(q)
    shape = (B, Tk, Hk, d)
    _need("q", q, q.shape, dt, dev, rows=True)
    _need("k", k, shape, dt, dev, rows=True)
    _need("v", v, shape, dt, dev, rows=True)
    if lens is not None:
        _need("lens", lens, (B,), torch.int32, dev)
    scale = d ** -0.5 if scale is None else float(scale)
    return B, T, Tk, Hq, Hk, d, int(window), int(sinks), scale, _strides(q, k, v), code, _raw_stream(dev)


def gdn2_swa_fwd(q, k, v, lens=None, o=None, lse=None, *, window, sinks=0, scale=None, want_lse=True, stream=None,
                 check=True):
    """Causal attention over a sliding window and ``sinks`` first tokens.  q [B,T,Hq,d], k and v
    [B,Tk,Hk,d] (Tk >= T; the queries are the last T positions), which may be strided views with
    contiguous rows, such as slices of one packed projection; ``lens`` [B] int32 or None; ``scale``
    defaults to d ** -0.5.  Returns (o, lse), lse [B,Hq,T] fp32 or None unless ``want_lse``."""
    dev = _here(q, stream)
    if dev < 0:
        return _there(gdn2_swa_fwd, stream, q, k, v, lens, o, lse, window=window, sinks=sinks, scale=scale,
                      want_lse=want_lse, check=check)
    args = _swa_sizes(q, k, v, lens, window, sinks, scale, dev)
    B, T, Hq, d = q.shape
    if o is None:
        o = torch.empty((B, T, Hq, d), dtype=q.dtype, device=q.device)
    else:
        _need("o", o, q.shape, q.dtype, dev)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device) if want_lse else None
    else:
        _need("lse", lse, (B, Hq, T), torch.float32, dev)
    st = _native().swa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lens), o.data_ptr(), _p(lse), *args)
    _done(st, check, "gdn2_swa_fwd")
    return o, lse


def gdn2_swa_bwd(q, k, v, o, lse, dO, lens=None, *, window, sinks=0, scale=None, stream=None, check=True):
    """Backward of gdn2_swa_fwd from its inputs, its o and lse, and dO [B,T,Hq,d]; returns a dict
    of dq, dk and dv (dense, in the inputs' dtype)."""
    dev = _here(q, stream)
    if dev < 0:
        return _there(gdn2_swa_bwd, stream, q, k, v, o, lse, dO, lens, window=window, sinks=sinks, scale=scale,
                      check=check)
    args = _swa_sizes(q, k, v, lens, window, sinks, scale, dev)
    B, T, Hq, d = q.shape
    _need("o", o, q.shape, q.dtype, dev)
    _need("dO", dO, q.shape, q.dtype, dev)
    _need("lse", lse, (B, Hq, T), torch.float32, dev)
    g = {n: torch.empty(t.shape, dtype=q.dtype, device=q.device) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    st = _native().swa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dO.data_ptr(),
                           _p(lens), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(), *args)
    _done(st, check, "gdn2_swa_bwd")
    return g


def gdn2_swa_decode(q, k, v, k_cache, v_cache, pos, o=None, *, window, sinks=0, scale=None, stream=None, check=True):
    """One token per sequence against a ring cache: q [B,Hq,d], new k and v [B,Hk,d] (all three may
    be strided views with contiguous rows), k_cache and v_cache [B,slots,Hk,d] updated in place, pos
    [B] int32 the new token's position (< 0: no sequence in this row).  Position p lives in slot p if
    p < sinks, else in slot sinks + (p - sinks) % (slots - sinks).  Returns o."""
    dev = _here(q, stream)
    if dev < 0:
        return _there(gdn2_swa_decode, stream, q, k, v, k_cache, v_cache, pos, o, window=window, sinks=sinks,
                      scale=scale, check=check)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B,Hq,d], the caches [B,slots,Hk,d]")
    B, Hq, d = q.shape
    cache = k_cache.shape
    _, slots, Hk, _ = cache
    dt, code = q.dtype, _code(q)
    row = (B, Hk, d)
    _need("q", q, q.shape, dt, dev, rows=True)
    _need("k", k, row, dt, dev, rows=True)
    _need("v", v, row, dt, dev, rows=True)
    _need("k_cache", k_cache, (B, slots, Hk, d), dt, dev)
    _need("v_cache", v_cache, cache, dt, dev)
    _need("pos", pos, (B,), torch.int32, dev)
    if o is None:
        o = torch.empty((B, Hq, d), dtype=dt, device=q.device)
    else:
        _need("o", o, q.shape, dt, dev)
    st = _native().swa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                              pos.data_ptr(), o.data_ptr(), B, slots, Hq, Hk, d, int(window), int(sinks),
                              d ** -0.5 if scale is None else float(scale), _strides(q, k, v), code, _raw_stream(dev))
    _done(st, check, "gdn2_swa_decode")
    return o


def gdn2_scan_fwd(x, w, log_alpha, h0=None, y=None, h_T=None, *, want_state=True, want_ckpt=False, stream=None,
                  check=True):
    """Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + w_t x_t per channel: x, w [B,T,C],
    log_alpha [B,T,C] fp32, h0 [B,C] fp32 or None.  Returns (y, h_T), and with ``want_ckpt``
    (y, h_T, ckpt), ckpt being what gdn2_scan_bwd needs."""
    dev = _here(x, stream)
    if dev < 0:
        return _there(gdn2_scan_fwd, stream, x, w, log_alpha, h0, y, h_T, want_state=want_state, want_ckpt=want_ckpt,
                      check=check)
    shape = x.shape
    B, T, C = shape
    dt, code = x.dtype, _code(x)
    _need("x", x, shape, dt, dev)
    _need("w", w, shape, dt, dev)
    _need("log_alpha", log_alpha, shape, torch.float32, dev)
    _need("h0", h0, (B, C), torch.float32, dev)
    _need("y", y, shape, dt, dev)
    _need("h_T", h_T, (B, C), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    if h_T is None and want_state:
        h_T = torch.empty((B, C), dtype=torch.float32, device=x.device)
    ckpt = None
    if want_ckpt:
        ckpt = torch.empty((B, -(-T // GDN2_SCAN_BLOCK), C), dtype=torch.float32, device=x.device)
    st = _native().scan_fwd(x.data_ptr(), w.data_ptr(), log_alpha.data_ptr(), _p(h0), y.data_ptr(), _p(h_T), _p(ckpt),
                            B, T, C, code, _raw_stream(dev))
    _done(st, check, "gdn2_scan_fwd")
    return (y, h_T, ckpt) if want_ckpt else (y, h_T)


def gdn2_scan_bwd(x, w, log_alpha, ckpt, dy, dh_T=None, *, want_dh0=True, stream=None, check=True):
    """Backward of gdn2_scan_fwd: its inputs and ckpt, dy [B,T,C] and dh_T [B,C] fp32 or None.
    Returns a dict of dx, dw (inputs' dtype), dlog_alpha and dh0 (fp32; dh0 None unless ``want_dh0``)."""
    dev = _here(x, stream)
    if dev < 0:
        return _there(gdn2_scan_bwd, stream, x, w, log_alpha, ckpt, dy, dh_T, want_dh0=want_dh0, check=check)
    shape = x.shape
    B, T, C = shape
    dt, code = x.dtype, _code(x)
    _need("x", x, shape, dt, dev)
    _need("w", w, shape, dt, dev)
    _need("log_alpha", log_alpha, shape, torch.float32, dev)
    _need("ckpt", ckpt, (B, -(-T // GDN2_SCAN_BLOCK), C), torch.float32, dev)
    _need("dy", dy, shape, dt, dev)
    _need("dh_T", dh_T, (B, C), torch.float32, dev)
    g = {"dx": torch.empty_like(x), "dw": torch.empty_like(x), "dlog_alpha": torch.empty_like(log_alpha),
         "dh0": torch.empty((B, C), dtype=torch.float32, device=x.device) if want_dh0 else None}
    st = _native().scan_bwd(x.data_ptr(), w.data_ptr(), log_alpha.data_ptr(), ckpt.data_ptr(), dy.data_ptr(), _p(dh_T),
                            g["dx"].data_ptr(), g["dw"].data_ptr(), g["dlog_alpha"].data_ptr(), _p(g["dh0"]),
                            B, T, C, code, _raw_stream(dev))
    _done(st, check, "gdn2_scan_bwd")
    return g


def gdn2_scan_step(x, w, log_alpha, h, y=None, *, stream=None, check=True):
    """One token of the recurrence: x, w [B,C], log_alpha and h [B,C] fp32, h updated in place.
    Returns y."""
    dev = _here(x, stream)
    if dev < 0:
        return _there(gdn2_scan_step, stream, x, w, log_alpha, h, y, check=check)
    shape = x.shape
    B, C = shape
    dt, code = x.dtype, _code(x)
    _need("x", x, shape, dt, dev)
    _need("w", w, shape, dt, dev)
    _need("log_alpha", log_alpha, shape, torch.float32, dev)
    _need("h", h, shape, torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need("y", y, shape, dt, dev)
    st = _native().scan_step(x.data_ptr(), w.data_ptr(), log_alpha.data_ptr(), h.data_ptr(), y.data_ptr(), B, C, code,
                             _raw_stream(dev))
    _done(st, check, "gdn2_scan_step")
    return y


def _norm_inputs(r, y, g_logit, w_post, res_scale, w_pre, dev):
    shape = r.shape
    D, dt, code = shape[-1], r.dtype, _code(r)
    _need("r", r, shape, dt, dev)
    _need("y", y, shape, dt, dev)
    _need("g_logit", g_logit, shape, dt, dev)
    _need("w_post", w_post, (D,), torch.float32, dev)
    _need("res_scale", res_scale, (D,), torch.float32, dev)
    _need("w_pre", w_pre, (D,), torch.float32, dev)
    return r.numel() // D if D else 0, D, code


def gdn2_block_norm_fwd(r, y, g_logit, w_post, res_scale, w_pre, eps=1e-6, r_out=None, x_out=None, *, stream=None,
                        check=True):
    """The norms around a block: r_out = r + res_scale * sigmoid(g_logit) * RMSNorm(y) * w_post and
    x_out = RMSNorm(r_out) * w_pre, over the last axis (r, y, g_logit of one shape; g_logit None: no
    gate; the three vectors fp32).  r_out may be r.  Returns (r_out, x_out)."""
    dev = _here(r, stream)
    if dev < 0:
        return _there(gdn2_block_norm_fwd, stream, r, y, g_logit, w_post, res_scale, w_pre, eps, r_out, x_out,
                      check=check)
    N, D, code = _norm_inputs(r, y, g_logit, w_post, res_scale, w_pre, dev)
    _need("r_out", r_out, r.shape, r.dtype, dev)
    _need("x_out", x_out, r.shape, r.dtype, dev)
    if r_out is None:
        r_out = torch.empty_like(r)
    if x_out is None:
        x_out = torch.empty_like(r)
    st = _native().block_norm_fwd(r.data_ptr(), y.data_ptr(), _p(g_logit), w_post.data_ptr(), res_scale.data_ptr(),
                                  w_pre.data_ptr(), eps, r_out.data_ptr(), x_out.data_ptr(), N, D, code,
                                  _raw_stream(dev))
    _done(st, check, "gdn2_block_norm_fwd")
    return r_out, x_out


def gdn2_block_norm_bwd(r, y, g_logit, w_post, res_scale, w_pre, dr_out, dx_out, eps=1e-6, *, stream=None,
                        check=True):
    """Backward of gdn2_block_norm_fwd from its inputs and the gradients of r_out and x_out.  Returns
    a dict of dr, dy, dg_logit (inputs' dtype; dg_logit None without a gate), dw_post, dres_scale and
    dw_pre (fp32)."""
    dev = _here(r, stream)
    if dev < 0:
        return _there(gdn2_block_norm_bwd, stream, r, y, g_logit, w_post, res_scale, w_pre, dr_out, dx_out, eps,
                      check=check)
    N, D, code = _norm_inputs(r, y, g_logit, w_post, res_scale, w_pre, dev)
    _need("dr_out", dr_out, r.shape, r.dtype, dev)
    _need("dx_out", dx_out, r.shape, r.dtype, dev)
    g = {"dr": torch.empty_like(r), "dy": torch.empty_like(r),
         "dg_logit": None if g_logit is None else torch.empty_like(r), "dw_post": torch.empty_like(w_post),
         "dres_scale": torch.empty_like(w_post), "dw_pre": torch.empty_like(w_post)}
    st = _native().block_norm_bwd(r.data_ptr(), y.data_ptr(), _p(g_logit), w_post.data_ptr(), res_scale.data_ptr(),
                                  w_pre.data_ptr(), eps, dr_out.data_ptr(), dx_out.data_ptr(), g["dr"].data_ptr(),
                                  g["dy"].data_ptr(), _p(g["dg_logit"]), g["dw_post"].data_ptr(),
                                  g["dres_scale"].data_ptr(), g["dw_pre"].data_ptr(), N, D, code, _raw_stream(dev))
    _done(st, check, "gdn2_block_norm_bwd")
    return g


def gdn2_check_device_error(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device error status."""
    return int(lib().gdn2_check_device_error(_stream(stream)))


def gdn2_selftest_bounded_wait(stream=None) -> int:
    """Queue the bounded-wait self-test (a wait that runs out after one second)."""
    return int(lib().gdn2_selftest_bounded_wait(_stream(stream)))


def gdn2_fwd_chunked_launches(B, T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Kernel launches one gdn2_fwd_chunked call makes for this problem."""
    code = GDN2_BF16 if dtype == torch.bfloat16 else GDN2_F32
    return int(lib().gdn2_fwd_chunked_launches(B, T, H, dk, dv, code))


def gdn2_status_string(status: int) -> str:
    return status_string(status)
