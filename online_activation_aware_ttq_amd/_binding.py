"""ctypes binding of ``libttq.so`` (the C ABI in ``include/ttq.h``).

Argument marshalling only: every step of the projection runs in the gfx950
kernels of the library.  Torch is used for device memory and streams.  If the
library has not been built, importing the compute functions raises -- there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# TTQ_LIBRARY selects another build of the same library (the CPU tests use
# it for a host build with address and undefined-behaviour sanitizers)
LIB_PATH = os.environ.get("TTQ_LIBRARY") or os.path.join(PKG_DIR, "libttq.so")

TTQ_OK = 0
TTQ_EINVAL = -1
TTQ_ENULL = -2
TTQ_EALIGN = -3
TTQ_EWORKSPACE = -4
TTQ_EUNSUPPORTED = -5
TTQ_EHIP = -100

TTQ_FLAG_FORCE_FUSED = 1
TTQ_FLAG_FORCE_TWO_PHASE = 2

# Every entry point include/ttq.h declares, with its ctypes signature.
_c = ctypes
_vp = _c.c_void_p
EXPORTS = {
    "ttq_workspace_bytes": (_c.c_int, [_vp, _c.c_int64, _c.POINTER(_c.c_size_t)]),
    "ttq_linear": (_c.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp, _c.c_size_t, _vp]),
    "ttq_linear_batched": (_c.c_int, [_vp, _c.c_int64, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _c.c_size_t,
                                      _vp]),
    "ttq_linear_noalloc": (_c.c_int, [_vp, _c.c_int64, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _vp]),
    "ttq_path": (_c.c_int, [_vp, _c.c_int64]),
    "ttq_segmented_workspace_bytes": (_c.c_int, [_vp, _c.c_int64, _vp,
                                                 _c.POINTER(_c.c_size_t)]),
    "ttq_linear_segmented": (_c.c_int, [_vp, _c.c_int64, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _c.c_size_t, _vp]),
    "ttq_packed_row_bytes": (_c.c_int, [_vp, _c.POINTER(_c.c_int64)]),
    "ttq_quantize_workspace_bytes": (_c.c_int, [_vp, _c.POINTER(_c.c_size_t)]),
    "ttq_qmatmul_workspace_bytes": (_c.c_int, [_vp, _c.POINTER(_c.c_size_t)]),
    "ttq_quantize": (_c.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _c.c_size_t, _vp]),
    "ttq_qmatmul": (_c.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _c.c_size_t, _vp]),
    "ttq_lowrank_pca_workspace_bytes": (_c.c_int, [_vp, _c.c_int32,
                                                   _c.POINTER(_c.c_size_t)]),
    "ttq_lowrank_pca": (_c.c_int, [_vp, _c.c_int32, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _c.c_size_t, _vp]),
    "ttq_adapters_workspace_bytes": (_c.c_int, [_vp, _c.c_int64,
                                                _c.POINTER(_c.c_size_t)]),
    "ttq_adapters": (_c.c_int, [_vp, _c.c_int64, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp, _c.c_size_t, _vp]),
    "ttq_moe_workspace_bytes": (_c.c_int, [_vp, _c.POINTER(_c.c_size_t)]),
    "ttq_moe": (_c.c_int, [_vp] * 15 + [_c.c_size_t, _vp]),
    "ttq_cache_write": (_c.c_int, [_vp, _c.c_int64, _c.c_int32, _vp, _c.c_int64,
                                   _vp, _vp, _vp, _vp, _vp, _vp]),
    "ttq_cache_read": (_c.c_int, [_vp, _c.c_int64, _c.c_int64, _c.c_int64,
                                  _c.c_int32, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _c.c_int32, _vp, _vp]),
    "ttq_status_string": (_c.c_char_p, [_c.c_int]),
    "ttq_last_hip_error": (_c.c_int, []),
    "ttq_stream_read": (_c.c_int, [_vp, _c.c_int64, _vp, _vp]),
    "ttq_version": (_c.c_char_p, []),
    "ttq_timing_enable": (_c.c_int, [_c.c_int]),
    "ttq_timing_reset": (_c.c_int, []),
    "ttq_kernel_count": (_c.c_int, []),
    "ttq_kernel_name": (_c.c_char_p, [_c.c_int]),
    "ttq_timing_query": (_c.c_int, [_c.c_int, _c.POINTER(_c.c_double),
                                    _c.POINTER(_c.c_int64)]),
}


class ttq_params(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int64),
        ("d_out", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("rank", ctypes.c_int64),
        ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("p", ctypes.c_double),
        ("lambda_", ctypes.c_double),
        ("alpha", ctypes.c_double),
        ("flags", ctypes.c_uint32),
        ("qformat", ctypes.c_uint32),
    ]


class ttq_moe_params(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("ff", ctypes.c_int64),
        ("experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("qformat", ctypes.c_uint32),
    ]


# quantizer formats (TTQ_QF_* of include/ttq.h)
QFORMATS = {"asym": 0, "sym": 1, "intzp": 2, "fp8": 3}


def qformat_code(qformat) -> int:
    """TTQ_QF_* value of a format name ("asym", "sym", "intzp", "fp8") or int."""
    if isinstance(qformat, str):
        if qformat not in QFORMATS:
            raise ValueError(f"unknown quantizer format {qformat!r}")
        return QFORMATS[qformat]
    return int(qformat)


class TTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = ttq_status_string(status)
        if status == TTQ_EHIP:
            msg += f" (hipError {load_library().ttq_last_hip_error()})"
        super().__init__(f"{where}: {msg} [{status}]")


_lib = None


def load_library() -> ctypes.CDLL:
    """Load the in-tree ``libttq.so``; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m online_activation_aware_ttq_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def make_params(*, d: int, d_out: int, T: int, rank: int = 0, bits: int,
                group: int, p: float, lam: float, alpha: float,
                flags: int = 0, qformat="asym") -> ttq_params:
    return ttq_params(int(d), int(d_out), int(T), int(rank), int(bits),
                      int(group), float(p), float(lam), float(alpha),
                      int(flags), qformat_code(qformat))


# The calls below build the same parameter block for every call of one shape;
# the library only reads it, so one block per shape is kept (bounded).
_PARAMS = {}


def _params(d, d_out, T, rank, bits, group, p, lam, alpha, flags, qformat):
    key = (d, d_out, T, rank, bits, group, p, lam, alpha, flags, qformat)
    prm = _PARAMS.get(key)
    if prm is None:
        if len(_PARAMS) > 4096:
            _PARAMS.clear()
            _NEED.clear()
        prm = _PARAMS[key] = make_params(d=d, d_out=d_out, T=T, rank=rank,
                                         bits=bits, group=group, p=p, lam=lam,
                                         alpha=alpha, flags=flags,
                                         qformat=qformat)
    return prm, key


# Looked up once: torch, its cheap accessor of the current stream's raw handle
# (where this torch build has it), and whether there are several devices.
_torch = None
_raw_stream = None
_several = None


def _host():
    global _torch, _raw_stream, _several
    import torch
    _several = torch.cuda.device_count() > 1
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _torch = torch
    return torch


def _current_stream(dev) -> int:
    """Raw handle of torch's current stream on `dev`."""
    torch = _torch or _host()
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


# Workspace for calls that bring none: one buffer per (thread, device, stream),
# kept between calls.  A thread's calls on one stream run in order, so they can
# share it; the kernels of two threads' calls may alternate on a stream, and calls
# on different streams run at once: those get different buffers.  A call that is
# being captured gets one of its own, which lives in the graph's memory: no other
# graph or call has it, and none is released under a graph.  (A capture that torch
# does not know of, by hipStreamBeginCapture, has no such memory: it has to bring
# its workspace.)  Buffers are taken as memory of the stream that uses them, where
# what was released is used again only behind the kernels enqueued before.
_NEED = {}


class _Scratch(threading.local):
    def __init__(self):
        self.kept = {}


_SCRATCH = _Scratch()


def _is_current(dev, stream):
    """Whether ``stream`` of ``dev`` is where torch allocates and enqueues now."""
    return stream == _current_stream(dev) and not (
        _several and dev.index != _torch.cuda.current_device())


def _scratch(torch, dev, stream, need):
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(need, dtype=torch.uint8, device=dev)
    kept, key = _SCRATCH.kept, (dev.index, stream)
    buf = kept.get(key)
    if buf is None or buf.numel() < need:
        buf = kept[key] = torch.empty(need, dtype=torch.uint8, device=dev)
    return buf


def _workspace(dev, stream, need_key, query, here=False):
    """A workspace of query() bytes, remembered by need_key (None: not); ``here``:
    the caller has just got ``stream`` as torch's current one."""
    torch = _torch or _host()
    need = _NEED.get(need_key) if need_key is not None else None
    if need is None:
        need = max(int(query()), 256)
        if need_key is not None:
            _NEED[need_key] = need
    if (here and not _several) or _is_current(dev, stream):
        return _scratch(torch, dev, stream, need)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
        return _scratch(torch, dev, stream, need)


def _result(shape, dtype, dev, stream, make=None):
    """Memory for a result of a call on ``stream`` (None: torch's current one),
    taken, and with ``make`` (torch.zeros) filled, there: in the order of that
    stream's work, and reused in it."""
    torch = _torch or _host()
    make = make or torch.empty
    if stream is None or _is_current(dev, stream):
        return make(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
        return make(shape, dtype=dtype, device=dev)


def ttq_status_string(status: int) -> str:
    return load_library().ttq_status_string(int(status)).decode()


def ttq_version() -> str:
    return load_library().ttq_version().decode()


def ttq_workspace_bytes(prm: ttq_params, n_requests: int = 1) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_workspace_bytes(ctypes.byref(prm), int(n_requests),
                                            ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_workspace_bytes")
    return int(out.value)


def ttq_path(prm: ttq_params, n_requests: int = 1) -> int:
    st = load_library().ttq_path(ctypes.byref(prm), int(n_requests))
    if st < 0:
        raise TTQError(st, "ttq_path")
    return st


# ------------------------------------------------------------------ torch side
def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t, name, dtype, shape, device):
    if t is None:
        return
    if getattr(t, "dtype", None) is not dtype:
        raise TypeError(f"{name} must be a torch.Tensor of {dtype}, got "
                        f"{getattr(t, 'dtype', type(t))}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _call(batched: bool, W, X, B, A, *, p, lam, alpha, bits, group, Y,
          codes_out, scales_out, mins_out, dhalf_out, workspace, stream,
          flags, qformat, noalloc=False):
    torch = _torch or _host()
    lib = load_library()
    if batched:
        R, T, d = X.shape
    else:
        (T, d), R = X.shape, 1
    d_out = W.shape[0]
    rank = 0 if A is None else A.shape[0]
    dev = W.device
    if dev.type != "cuda":
        raise ValueError("W must be a GPU tensor")
    lead = (R,) if batched else ()
    G = d // group if group > 0 and d % group == 0 else 0
    _check(W, "W", torch.bfloat16, (d_out, d), dev)
    _check(X, "X", torch.bfloat16, lead + (T, d), dev)
    _check(B, "B", torch.bfloat16, (d_out, rank), dev)
    _check(A, "A", torch.bfloat16, (rank, d), dev)
    if (A is None) != (B is None):
        raise ValueError("pass both B and A or neither")
    prm, key = _params(d, d_out, T, rank, bits, group, p, lam, alpha, flags,
                       qformat)
    if Y is None:
        Y = _result(lead + (T, d_out), torch.float32, dev, stream)
    _check(Y, "Y", torch.float32, lead + (T, d_out), dev)
    _check(codes_out, "codes_out", torch.uint8, lead + (d_out, d), dev)
    _check(scales_out, "scales_out", torch.float32, lead + (d_out, G), dev)
    _check(mins_out, "mins_out", torch.float32, lead + (d_out, G), dev)
    _check(dhalf_out, "dhalf_out", torch.float32, lead + (d,), dev)
    here = stream is None
    if here:
        stream = _current_stream(dev)
    if noalloc:
        args = [_ptr(W), _ptr(X), _ptr(B), _ptr(A), _ptr(Y), _ptr(codes_out),
                _ptr(scales_out), _ptr(mins_out), _ptr(dhalf_out), stream]
        st = lib.ttq_linear_noalloc(ctypes.byref(prm), R, *args)
        if st != TTQ_OK:
            raise TTQError(st, "ttq_linear_noalloc")
        return Y
    if workspace is None:  # (a given workspace is checked by the library)
        workspace = _workspace(dev, stream, ("linear", key, R),
                               lambda: ttq_workspace_bytes(prm, R), here)
    args = [_ptr(W), _ptr(X), _ptr(B), _ptr(A), _ptr(Y), _ptr(codes_out),
            _ptr(scales_out), _ptr(mins_out), _ptr(dhalf_out),
            _ptr(workspace), workspace.numel(), stream]
    if batched:
        st = lib.ttq_linear_batched(ctypes.byref(prm), R, *args)
    else:
        st = lib.ttq_linear(ctypes.byref(prm), *args)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_linear_batched" if batched else "ttq_linear")
    return Y


def ttq_linear(W, X, B=None, A=None, *, p: float, lam: float, alpha: float,
               bits: int, group: int, Y=None, codes_out=None, scales_out=None,
               mins_out=None, dhalf_out=None, workspace=None, stream=None,
               flags: int = 0, qformat="asym"):
    """Y[T, d_out] = Q_D[W] X + B (A X) for one request (see include/ttq.h).

    W [d_out, d], X [T, d], B [d_out, r], A [r, d] are bfloat16 GPU tensors;
    Y is float32.  Enqueued on ``stream`` (default: torch's current stream); the
    results that this and the other calls make are memory of that stream, as if
    made under ``torch.cuda.stream``.
    """
    return _call(False, W, X, B, A, p=p, lam=lam, alpha=alpha, bits=bits,
                 group=group, Y=Y, codes_out=codes_out, scales_out=scales_out,
                 mins_out=mins_out, dhalf_out=dhalf_out, workspace=workspace,
                 stream=stream, flags=flags, qformat=qformat)


def ttq_linear_batched(W, X, B=None, A=None, *, p: float, lam: float,
                       alpha: float, bits: int, group: int, Y=None,
                       codes_out=None, scales_out=None, mins_out=None,
                       dhalf_out=None, workspace=None, stream=None,
                       flags: int = 0, qformat="asym"):
    """R requests with their own statistics on a shared W: X [R, T, d]."""
    return _call(True, W, X, B, A, p=p, lam=lam, alpha=alpha, bits=bits,
                 group=group, Y=Y, codes_out=codes_out, scales_out=scales_out,
                 mins_out=mins_out, dhalf_out=dhalf_out, workspace=workspace,
                 stream=stream, flags=flags, qformat=qformat)


def ttq_linear_noalloc(W, X, B=None, A=None, *, p: float, lam: float,
                       alpha: float, bits: int, group: int, Y,
                       codes_out=None, scales_out=None, mins_out=None,
                       dhalf_out=None, stream=None, flags: int = 0,
                       qformat="asym"):
    """ttq_linear_batched (X [R, T, d]) on the library's static scratch: no
    workspace and no allocation; Y must be given (see include/ttq.h)."""
    if Y is None:
        raise ValueError("ttq_linear_noalloc needs a preallocated Y")
    return _call(True, W, X, B, A, p=p, lam=lam, alpha=alpha, bits=bits,
                 group=group, Y=Y, codes_out=codes_out, scales_out=scales_out,
                 mins_out=mins_out, dhalf_out=dhalf_out, workspace=None,
                 stream=stream, flags=flags, qformat=qformat, noalloc=True)


TTQ_NOALLOC_SCRATCH_BYTES = 64 << 20


def _offsets(seg_offsets):
    arr = (ctypes.c_int64 * len(seg_offsets))(*[int(v) for v in seg_offsets])
    return arr, len(seg_offsets) - 1


def ttq_segmented_workspace_bytes(prm: ttq_params, seg_offsets) -> int:
    arr, n = _offsets(seg_offsets)
    out = ctypes.c_size_t(0)
    st = load_library().ttq_segmented_workspace_bytes(
        ctypes.byref(prm), n, ctypes.cast(arr, ctypes.c_void_p), ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_segmented_workspace_bytes")
    return int(out.value)


def ttq_linear_segmented(W, X, B=None, A=None, *, seg_offsets, p: float,
                         lam: float, alpha: float, bits: int, group: int,
                         Y=None, codes_out=None, scales_out=None, mins_out=None,
                         dhalf_out=None, workspace=None, stream=None,
                         flags: int = 0, qformat="asym"):
    """Requests of different lengths packed in X [T, d]: request i owns rows
    seg_offsets[i] .. seg_offsets[i+1]-1 and has its own statistics."""
    torch = _torch or _host()
    T, d = X.shape
    d_out = W.shape[0]
    rank = 0 if A is None else A.shape[0]
    dev = W.device
    if dev.type != "cuda":
        raise ValueError("W must be a GPU tensor")
    n = len(seg_offsets) - 1
    G = d // group if group > 0 and d % group == 0 else 0
    _check(W, "W", torch.bfloat16, (d_out, d), dev)
    _check(X, "X", torch.bfloat16, (T, d), dev)
    _check(B, "B", torch.bfloat16, (d_out, rank), dev)
    _check(A, "A", torch.bfloat16, (rank, d), dev)
    if (A is None) != (B is None):
        raise ValueError("pass both B and A or neither")
    prm = make_params(d=d, d_out=d_out, T=T, rank=rank, bits=bits,
                      group=group, p=p, lam=lam, alpha=alpha, flags=flags,
                      qformat=qformat)
    if Y is None:
        Y = _result((T, d_out), torch.float32, dev, stream)
    _check(Y, "Y", torch.float32, (T, d_out), dev)
    _check(codes_out, "codes_out", torch.uint8, (n, d_out, d), dev)
    _check(scales_out, "scales_out", torch.float32, (n, d_out, G), dev)
    _check(mins_out, "mins_out", torch.float32, (n, d_out, G), dev)
    _check(dhalf_out, "dhalf_out", torch.float32, (n, d), dev)
    if stream is None:
        stream = _current_stream(dev)
    if workspace is None:
        workspace = _workspace(dev, stream, None,
                               lambda: ttq_segmented_workspace_bytes(prm, seg_offsets))
    arr, _ = _offsets(seg_offsets)
    st = load_library().ttq_linear_segmented(
        ctypes.byref(prm), n, ctypes.cast(arr, ctypes.c_void_p), _ptr(W),
        _ptr(X), _ptr(B), _ptr(A), _ptr(Y), _ptr(codes_out), _ptr(scales_out),
        _ptr(mins_out), _ptr(dhalf_out), _ptr(workspace), workspace.numel(),
        stream)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_linear_segmented")
    return Y


# ------------------------------------------- quantize once, decode from codes
def container_bits(bits: int) -> int:
    """Bits each stored code takes (1, 2, 4 or 8)."""
    return 1 if bits <= 1 else 2 if bits <= 2 else 4 if bits <= 4 else 8


def ttq_packed_row_bytes(prm: ttq_params) -> int:
    out = ctypes.c_int64(0)
    st = load_library().ttq_packed_row_bytes(ctypes.byref(prm), ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_packed_row_bytes")
    return int(out.value)


_ROW_BYTES = {}


def _row_bytes(d: int, bits: int, group: int) -> int:
    """Packed row bytes for the shape checks of the calls below (the calls
    themselves validate every parameter)."""
    key = (d, bits, group)
    if key not in _ROW_BYTES:
        _ROW_BYTES[key] = ttq_packed_row_bytes(
            make_params(d=d, d_out=1, T=0, bits=bits, group=group, p=1.0,
                        lam=0.0, alpha=0.0))
    return _ROW_BYTES[key]


def ttq_quantize_workspace_bytes(prm: ttq_params) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_quantize_workspace_bytes(ctypes.byref(prm),
                                                     ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_quantize_workspace_bytes")
    return int(out.value)


def ttq_qmatmul_workspace_bytes(prm: ttq_params) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_qmatmul_workspace_bytes(ctypes.byref(prm),
                                                    ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_qmatmul_workspace_bytes")
    return int(out.value)


def ttq_quantize(W, X, *, p: float, lam: float, alpha: float, bits: int,
                 group: int, codes=None, scales=None, mins=None,
                 dhalf_inv=None, dhalf_out=None, workspace=None, stream=None,
                 qformat="asym"):
    """Quantize W once for the prompt X (see include/ttq.h).

    Returns (codes [d_out, row_bytes] uint8, scales [d_out, G] float32,
    mins [d_out, G] float32, dhalf_inv [d] float32).
    """
    torch = _torch or _host()
    lib = load_library()
    T, d = X.shape
    d_out = W.shape[0]
    dev = W.device
    if dev.type != "cuda":
        raise ValueError("W must be a GPU tensor")
    prm = make_params(d=d, d_out=d_out, T=T, bits=bits, group=group, p=p,
                      lam=lam, alpha=alpha, qformat=qformat)
    rb = ttq_packed_row_bytes(prm)
    G = d // group
    _check(W, "W", torch.bfloat16, (d_out, d), dev)
    _check(X, "X", torch.bfloat16, (T, d), dev)
    if codes is None:
        codes = _result((d_out, rb), torch.uint8, dev, stream)
    if scales is None:
        scales = _result((d_out, G), torch.float32, dev, stream)
    if mins is None:
        mins = _result((d_out, G), torch.float32, dev, stream)
    if dhalf_inv is None:
        dhalf_inv = _result((d,), torch.float32, dev, stream)
    _check(codes, "codes", torch.uint8, (d_out, rb), dev)
    _check(scales, "scales", torch.float32, (d_out, G), dev)
    _check(mins, "mins", torch.float32, (d_out, G), dev)
    _check(dhalf_inv, "dhalf_inv", torch.float32, (d,), dev)
    _check(dhalf_out, "dhalf_out", torch.float32, (d,), dev)
    if stream is None:
        stream = _current_stream(dev)
    if workspace is None:
        workspace = _workspace(dev, stream, None,
                               lambda: ttq_quantize_workspace_bytes(prm))
    st = lib.ttq_quantize(ctypes.byref(prm), _ptr(W), _ptr(X), _ptr(codes),
                          _ptr(scales), _ptr(mins), _ptr(dhalf_inv),
                          _ptr(dhalf_out), _ptr(workspace), workspace.numel(),
                          stream)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_quantize")
    return codes, scales, mins, dhalf_inv


def ttq_qmatmul(codes, scales, mins, dhalf_inv, X, B=None, A=None, *,
                bits: int, group: int, Y=None, workspace=None, stream=None,
                flags: int = 0, qformat="asym"):
    """Y[T, d_out] = X ((min + s q) D^{-1/2})^T + (X A^T) B^T from the codes
    stored by ttq_quantize (see include/ttq.h; ``qformat`` as given to it:
    E4M3 codes decode as FP8 values)."""
    torch = _torch or _host()
    lib = load_library()
    T, d = X.shape
    d_out = codes.shape[0]
    rank = 0 if A is None else A.shape[0]
    dev = X.device
    if dev.type != "cuda":
        raise ValueError("X must be a GPU tensor")
    if (A is None) != (B is None):
        raise ValueError("pass both B and A or neither")
    prm, key = _params(d, d_out, T, rank, bits, group, 1.0, 0.0, 0.0, flags,
                       qformat)
    rb = _row_bytes(d, bits, group)
    G = d // group
    _check(codes, "codes", torch.uint8, (d_out, rb), dev)
    _check(scales, "scales", torch.float32, (d_out, G), dev)
    _check(mins, "mins", torch.float32, (d_out, G), dev)
    _check(dhalf_inv, "dhalf_inv", torch.float32, (d,), dev)
    _check(X, "X", torch.bfloat16, (T, d), dev)
    _check(B, "B", torch.bfloat16, (d_out, rank), dev)
    _check(A, "A", torch.bfloat16, (rank, d), dev)
    if Y is None:
        Y = _result((T, d_out), torch.float32, dev, stream)
    _check(Y, "Y", torch.float32, (T, d_out), dev)
    here = stream is None
    if here:
        stream = _current_stream(dev)
    if workspace is None:  # (a given workspace is checked by the library)
        workspace = _workspace(dev, stream, ("qmatmul", key),
                               lambda: ttq_qmatmul_workspace_bytes(prm), here)
    st = lib.ttq_qmatmul(ctypes.byref(prm), _ptr(codes), _ptr(scales),
                         _ptr(mins), _ptr(dhalf_inv), _ptr(X), _ptr(B), _ptr(A),
                         _ptr(Y), _ptr(workspace), workspace.numel(), stream)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_qmatmul")
    return Y


# --------------------------------------------- one decode step from codes
TTQ_BF16 = 0
TTQ_F32 = 1
TTQ_MOE_RENORMALIZE = 1


def _elem_type(t, name) -> int:
    torch = _torch or _host()
    dt = getattr(t, "dtype", None)
    if dt is torch.bfloat16:
        return TTQ_BF16
    if dt is torch.float32:
        return TTQ_F32
    raise TypeError(f"{name} must be a torch.Tensor of torch.bfloat16 or "
                    f"torch.float32, got {dt if dt is not None else type(t)}")


# A decode step makes many small calls, so these entry points keep their host
# time short: what a shape implies (parameter block, expected types and shapes,
# workspace need) is worked out once per shape, and a call only compares.
_PLANS = {}


def _plan(key, make):
    plan = _PLANS.get(key)
    if plan is None:
        if len(_PLANS) > 4096:
            _PLANS.clear()
        plan = _PLANS[key] = make()
    return plan


def _expect(tensors, want, dev):
    """Raise unless every tensor (None: absent) is as its (name, dtype, shape)
    says (shape None: part of the plan's key), contiguous and on ``dev``; returns
    their addresses."""
    di = dev.index
    ptrs = []
    for t, (name, dtype, shape) in zip(tensors, want):
        if t is None:
            ptrs.append(None)
            continue
        try:
            ok = (t.dtype is dtype and (shape is None or t.shape == shape)
                  and t.get_device() == di and t.is_contiguous())
        except AttributeError:
            ok = False
        if not ok:
            _check(t, name, dtype, t.shape if shape is None else shape, dev)
        ptrs.append(t.data_ptr())
    return ptrs


# Entry points, looked up once.
_lib_fn = {}


def _enqueue(where, dev, *args):
    """Call a library entry point with the tensors' device current."""
    fn = _lib_fn.get(where)
    if fn is None:
        fn = _lib_fn[where] = getattr(load_library(), where)
    if _several and dev.index != _torch.cuda.current_device():
        with _torch.cuda.device(dev):
            st = fn(*args)
    else:
        st = fn(*args)
    if st != TTQ_OK:
        raise TTQError(st, where)


def _gpu(t, name):
    """Device of ``t``, which has to be a GPU tensor."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    return dev


def _step_workspace(dev, stream, need, given, here=False):
    """The caller's workspace, or one of ``need`` bytes (see _workspace)."""
    if given is not None:
        if given.dtype is not _torch.uint8:
            raise TypeError(f"workspace must be a torch.Tensor of torch.uint8, got {given.dtype}")
        if given.device != dev or not given.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {dev}, got {given.device}")
        return given
    if here and not _several:
        return _scratch(_torch, dev, stream, need)
    return _workspace(dev, stream, None, lambda: need)


def ttq_adapters_workspace_bytes(prm: ttq_params, n_adapters: int) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_adapters_workspace_bytes(
        ctypes.byref(prm), int(n_adapters), ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_adapters_workspace_bytes")
    return int(out.value)


def ttq_adapters(X, A, B, index, *, scale=None, base=None, Y=None,
                 workspace=None, stream=None):
    """Y[t] = base[t] + scale[e] B[e] (A[e] x_t) with e = index[t]: low-rank
    adapters of many requests beside a shared projection (see include/ttq.h).

    X [T, d], A [n, r, d] and B [n, d_out, r] are bfloat16, ``scale`` [n] and
    ``base`` [T, d_out] float32, ``index`` [T] int32 (outside 0 .. n - 1: no
    pair).  ``base`` is what ttq_linear, ttq_linear_batched (flattened),
    ttq_linear_segmented or ttq_qmatmul gave for X; ``Y=base`` adds in place.
    """
    torch = _torch or _host()
    xs, as_, bs = X.shape, A.shape, B.shape
    dev = _gpu(X, "X")

    def make():
        (T, d), (n, r, _), d_out = xs, as_, bs[1]
        bf, f32 = torch.bfloat16, torch.float32
        _check(A, "A", bf, (n, r, d), dev)
        _check(B, "B", bf, (n, d_out, r), dev)
        prm = make_params(d=d, d_out=d_out, T=T, rank=r, bits=4, group=32, p=2.0,
                          lam=0.0, alpha=0.0)
        return n, (T, d_out), ctypes.byref(prm), ttq_adapters_workspace_bytes(prm, n), (
            ("X", bf, None), ("A", bf, None), ("B", bf, None),
            ("scale", f32, (n,)), ("index", torch.int32, (T,)),
            ("base", f32, (T, d_out)), ("Y", f32, (T, d_out)))

    n, ys, prm, need, want = _plan(("adapters", xs, as_, bs), make)
    if Y is None:
        Y = _result(ys, torch.float32, dev, stream)
    ptrs = _expect((X, A, B, scale, index, base, Y), want, dev)
    here = stream is None
    if here:
        stream = _current_stream(dev)
    ws = size = 0
    if need or workspace is not None:  # (small steps need none)
        workspace = _step_workspace(dev, stream, need, workspace, here)
        ws, size = workspace.data_ptr(), workspace.numel()
    _enqueue("ttq_adapters", dev, prm, n, *ptrs, ws, size, stream)
    return Y


def make_moe_params(*, T: int, d: int, ff: int, experts: int, top_k: int,
                    bits: int, group: int, renormalize: bool = True,
                    qformat="asym") -> ttq_moe_params:
    return ttq_moe_params(int(T), int(d), int(ff), int(experts), int(top_k),
                          int(bits), int(group),
                          TTQ_MOE_RENORMALIZE if renormalize else 0,
                          qformat_code(qformat))


def ttq_moe_workspace_bytes(prm: ttq_moe_params) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_moe_workspace_bytes(ctypes.byref(prm), ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_moe_workspace_bytes")
    return int(out.value)


def ttq_moe(X, router, gu_codes, gu_scales, gu_mins, gu_dhalf_inv, dn_codes,
            dn_scales, dn_mins, dn_dhalf_inv, *, top_k: int, bits: int,
            group: int, renormalize: bool = True, Y=None, ids_out=None,
            weights_out=None, workspace=None, stream=None, qformat="asym"):
    """Y[T, d] = a mixture-of-experts layer for a few tokens X [T, d], its
    experts' projections being codes stored by ttq_quantize (see
    include/ttq.h): gate rows followed by up rows in gu_* [E, 2 ff, ...], down
    rows in dn_* [E, d, ...], dhalf_inv [E, d] and [E, ff]; router [E, d]
    bfloat16.  ``ids_out`` and ``weights_out`` [T, top_k] receive the chosen
    experts (int32, best first) and their weights (float32)."""
    torch = _torch or _host()
    xs, es = X.shape, dn_dhalf_inv.shape
    dev = _gpu(X, "X")

    def make():
        (T, d), (E, ff) = xs, es
        prm = make_moe_params(T=T, d=d, ff=ff, experts=E, top_k=top_k, bits=bits,
                              group=group, renormalize=renormalize,
                              qformat=qformat)
        need = max(256, ttq_moe_workspace_bytes(prm))
        bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        rb, rf = (_row_bytes(c, bits, group) for c in (d, ff))
        gu, dn = (E, 2 * ff, d // group), (E, d, ff // group)
        return (T, d), ctypes.byref(prm), need, (
            ("X", bf, None), ("router", bf, (E, d)),
            ("gu_codes", u8, (E, 2 * ff, rb)), ("gu_scales", f32, gu),
            ("gu_mins", f32, gu), ("gu_dhalf_inv", f32, (E, d)),
            ("dn_codes", u8, (E, d, rf)), ("dn_scales", f32, dn),
            ("dn_mins", f32, dn), ("dn_dhalf_inv", f32, None),
            ("Y", f32, (T, d)), ("ids_out", torch.int32, (T, top_k)),
            ("weights_out", f32, (T, top_k)))

    ys, prm, need, want = _plan(("moe", xs, es, top_k, bits, group,
                                 bool(renormalize), qformat), make)
    if Y is None:
        Y = _result(ys, torch.float32, dev, stream)
    ptrs = _expect((X, router, gu_codes, gu_scales, gu_mins, gu_dhalf_inv,
                    dn_codes, dn_scales, dn_mins, dn_dhalf_inv, Y, ids_out,
                    weights_out), want, dev)
    here = stream is None
    if here:
        stream = _current_stream(dev)
    workspace = _step_workspace(dev, stream, need, workspace, here)
    _enqueue("ttq_moe", dev, prm, *ptrs, workspace.data_ptr(), workspace.numel(),
             stream)
    return Y


def _cache_params(T, d, bits, group, qformat):
    """Parameter block and packed row bytes of a cache of d channels."""
    prm = make_params(d=d, d_out=1, T=T, bits=bits, group=group, p=2.0, lam=0.0,
                      alpha=0.0, qformat=qformat)
    return prm, ttq_packed_row_bytes(prm)


def ttq_cache_write(X, slots, codes, scales, mins, *, bits: int, group: int,
                    dhalf=None, qformat="asym", stream=None):
    """Quantize the rows of X [T, d] (bfloat16 or float32; rows may lie apart,
    e.g. the K and V columns of a wider matrix) into the cache rows
    ``slots`` [T] (int64; a negative one is padding and not written).

    The cache is (codes [n_slots, row_bytes] uint8, scales and mins [n_slots,
    d / group] float32), updated in place; with ``dhalf`` [d] the codes are
    those of x D^{1/2} (see include/ttq.h).
    """
    torch = _torch or _host()
    xs, cs = X.shape, codes.shape
    dev = _gpu(codes, "codes")
    x_type = _elem_type(X, "X")
    if X.get_device() != dev.index:
        raise ValueError(f"X must be on {dev}, got {X.device}")
    ld, one = X.stride()
    T, d = xs
    if d > 1 and one != 1:
        raise ValueError("X must have contiguous rows")
    ldx = ld if T > 1 else d

    def make():
        f32, n_slots = torch.float32, cs[0]
        prm, rb = _cache_params(T, d, bits, group, qformat)
        _check(codes, "codes", torch.uint8, (n_slots, rb), dev)
        return n_slots, ctypes.byref(prm), (
            ("dhalf", f32, (d,)), ("slots", torch.int64, (T,)),
            ("codes", torch.uint8, None),
            ("scales", f32, (n_slots, d // group)),
            ("mins", f32, (n_slots, d // group)))

    n_slots, prm, want = _plan(("write", xs, cs, bits, group, qformat), make)
    ptrs = _expect((dhalf, slots, codes, scales, mins), want, dev)
    if stream is None:
        stream = _current_stream(dev)
    _enqueue("ttq_cache_write", dev, prm, n_slots, x_type, X.data_ptr(), ldx,
             *ptrs, stream)


def ttq_cache_read(codes, scales, mins, pages, lens, *, bits: int, group: int,
                   page_tokens: int, out=None, T=None, d=None, dhalf_inv=None,
                   dtype=None, qformat="asym", stream=None):
    """Read sequences back from a cache: out [n_seq, T, d] (bfloat16 or
    float32), row t of sequence i from page ``pages[i, t // page_tokens]``.

    ``pages`` [n_seq, max_pages] and ``lens`` [n_seq] are int32.  Rows behind a
    sequence's length are left as they were; without ``out`` a tensor of zeros
    for ``T`` rows of ``d`` channels is made (default: all pages, the channels
    of the stored groups; ``dtype`` bfloat16 by default).
    """
    torch = _torch or _host()
    ps, cs = pages.shape, codes.shape
    dev = _gpu(codes, "codes")
    if out is None:
        d = scales.shape[1] * group if d is None else d
        T = ps[1] * page_tokens if T is None else T
        out = _result((ps[0], T, d), dtype or torch.bfloat16, dev, stream, torch.zeros)
    os_ = out.shape
    out_type = _elem_type(out, "out")

    def make():
        (n_seq, max_pages), n_slots, (_, T, d) = ps, cs[0], os_
        f32, i32 = torch.float32, torch.int32
        prm, rb = _cache_params(T, d, bits, group, qformat)
        _check(codes, "codes", torch.uint8, (n_slots, rb), dev)
        _check(out, "out", (torch.bfloat16, f32)[out_type], (n_seq, T, d), dev)
        return n_slots, n_seq, max_pages, ctypes.byref(prm), (
            ("pages", i32, None), ("lens", i32, (n_seq,)),
            ("codes", torch.uint8, None),
            ("scales", f32, (n_slots, d // group)),
            ("mins", f32, (n_slots, d // group)), ("dhalf_inv", f32, (d,)),
            ("out", (torch.bfloat16, f32)[out_type], None))

    n_slots, n_seq, max_pages, prm, want = _plan(
        ("read", ps, cs, os_, out_type, bits, group, qformat), make)
    *ptrs, po = _expect((pages, lens, codes, scales, mins, dhalf_inv, out), want,
                        dev)
    if stream is None:
        stream = _current_stream(dev)
    _enqueue("ttq_cache_read", dev, prm, n_slots, n_seq, max_pages, page_tokens,
             *ptrs, out_type, po, stream)
    return out


# ------------------------------------------------- low-rank factors by PCA
def ttq_lowrank_pca_workspace_bytes(prm: ttq_params, iters: int) -> int:
    out = ctypes.c_size_t(0)
    st = load_library().ttq_lowrank_pca_workspace_bytes(
        ctypes.byref(prm), int(iters), ctypes.byref(out))
    if st != TTQ_OK:
        raise TTQError(st, "ttq_lowrank_pca_workspace_bytes")
    return int(out.value)


def ttq_lowrank_pca(W, Omega, *, iters: int, X=None, p: float = 2.0,
                    lam: float = 0.0, alpha: float = 0.0, want_residual=True,
                    workspace=None, stream=None):
    """Low-rank factors by PCA (see include/ttq.h): returns (B [d_out, r],
    A [r, d], Wres [d_out, d] or None), bf16 GPU tensors.  ``Omega`` is the
    float32 [d, r] Gaussian test matrix; with ``X`` ([T, d] bf16) the
    principal subspace is that of W D^{1/2}."""
    torch = _torch or _host()
    d_out, d = W.shape
    r = Omega.shape[1]
    T = 0 if X is None else X.shape[0]
    dev = W.device
    if dev.type != "cuda":
        raise ValueError("W must be a GPU tensor")
    _check(W, "W", torch.bfloat16, (d_out, d), dev)
    _check(Omega, "Omega", torch.float32, (d, r), dev)
    if X is not None:
        _check(X, "X", torch.bfloat16, (T, d), dev)
    prm = make_params(d=d, d_out=d_out, T=T, rank=r, bits=4, group=32, p=p,
                      lam=lam, alpha=alpha)
    B = _result((d_out, r), torch.bfloat16, dev, stream)
    A = _result((r, d), torch.bfloat16, dev, stream)
    Wres = _result((d_out, d), torch.bfloat16, dev, stream) if want_residual else None
    if stream is None:
        stream = _current_stream(dev)
    if workspace is None:
        workspace = _workspace(dev, stream, None,
                               lambda: ttq_lowrank_pca_workspace_bytes(prm, iters))
    st = load_library().ttq_lowrank_pca(
        ctypes.byref(prm), int(iters), _ptr(W), _ptr(X), _ptr(Omega), _ptr(B),
        _ptr(A), _ptr(Wres), _ptr(workspace), workspace.numel(), stream)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_lowrank_pca")
    return B, A, Wres


# ------------------------------------------------------------------ timing
def stream_read(src, sink=None, stream=None):
    """Plain read of a device tensor's bytes (the ceiling of a one-pass
    kernel over W; see ttq_stream_read).  Returns the per-workgroup XOR
    words (uint32 stored in an int32 tensor)."""
    torch = _torch or _host()
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("stream_read: src must be a contiguous device tensor")
    nbytes = src.numel() * src.element_size()
    nblk = -(-nbytes // (128 * 1024))
    if sink is None:
        sink = _result(max(1, nblk), torch.int32, src.device, stream)
    if stream is None:
        stream = _current_stream(src.device)
    st = load_library().ttq_stream_read(_ptr(src), nbytes, _ptr(sink), stream)
    if st != TTQ_OK:
        raise TTQError(st, "ttq_stream_read")
    return sink


def timing_enable(on: bool = True) -> None:
    load_library().ttq_timing_enable(1 if on else 0)


def timing_reset() -> None:
    load_library().ttq_timing_reset()


def timing_query() -> dict:
    """{kernel name: (total milliseconds, launches)} for recorded launches."""
    lib = load_library()
    out = {}
    for k in range(lib.ttq_kernel_count()):
        ms = ctypes.c_double(0.0)
        n = ctypes.c_int64(0)
        st = lib.ttq_timing_query(k, ctypes.byref(ms), ctypes.byref(n))
        if st != TTQ_OK:
            raise TTQError(st, "ttq_timing_query")
        out[lib.ttq_kernel_name(k).decode()] = (ms.value, n.value)
    return out
