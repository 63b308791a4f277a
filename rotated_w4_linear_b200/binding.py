"""Thin ctypes binding of libparo.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: tensors are checked for dtype/device/contiguity and
their data pointers are handed to the library together with torch's current
CUDA stream. If the library is missing the import fails loudly; there is no
fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libparo.so")

PARO_OK = 0
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # paro_act
_STATUS = {0: "PARO_OK", 1: "PARO_ERR_ARG", 2: "PARO_ERR_UNSUPPORTED", 3: "PARO_ERR_CUDA", 4: "PARO_ERR_DEVICE"}

_lib: Optional[ctypes.CDLL] = None

_vp, _i64, _int, _sz, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "paro_rot_create": [ctypes.POINTER(_vp), _i64, _int, _int, _int, _vp, _vp, _vp],
    "paro_rot_destroy": [_vp],
    "paro_rotate": [_vp, _vp, _vp, _i64, _vp],
    "paro_pack_size": [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)],
    "paro_pack_weights": [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp],
    "paro_dequant": [_vp, _vp, _vp, _i64, _i64, _vp, _vp],
    "paro_quantize_weights": [_vp, _vp, _i64, _vp, _vp, _vp, _vp],
    "paro_linear_workspace_size": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "paro_linear": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_linear_bias": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_linear_noalloc": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp],
    "paro_pack_size_ex": [_i64, _i64, _int, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)],
    "paro_pack_weights_ex": [_vp, _vp, _vp, _i64, _i64, _int, _vp, _vp, _vp, _vp],
    "paro_dequant_ex": [_vp, _vp, _vp, _i64, _i64, _int, _vp, _vp],
    "paro_linear_ex": [_vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_linear_partial": [_vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_finalize": [_vp, _vp, _vp, _i64, _i64, _vp],
    "paro_linear_act": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_pack_gated": [_vp, _vp, _vp, _i64, _i64, _int, _vp, _vp, _vp, _vp],
    "paro_linear_gated": [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _vp, _i64, _i64, _i64, _vp, _sz, _vp],
    "paro_rmsnorm": [_vp, _int, _vp, _vp, _vp, _f32, _vp, _vp, _i64, _i64, _vp],
    "paro_rmsnorm_q8": [_vp, _int, _vp, _vp, _vp, _f32, _int, _vp, _vp, _vp, _i64, _i64, _vp],
    "paro_q8_expand": [_vp, _vp, _int, _vp, _i64, _i64, _vp],
    "paro_rotate_once": [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _int, _int, _int, _vp],
    "paro_linear_once": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp],
    "paro_fault_status": [ctypes.POINTER(_int), _int],
    "paro_check_wait_timeout": [ctypes.c_uint32, _vp],
    "paro_last_error": [],
}


class ParoError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libparo.so (built in-tree by rotated_w4_linear_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m rotated_w4_linear_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_char_p if name == "paro_last_error" else ctypes.c_int
        _lib = L
    return _lib


def _check(fn: str, st: int) -> None:
    if st != PARO_OK:
        raise ParoError(fn, st, lib().paro_last_error().decode())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: Optional[torch.device] = None) -> int:
    """Raw cudaStream_t: the given stream, else the current stream of the
    tensor's device (read without building a torch Stream object, which
    costs a few microseconds per call on the decode path)."""
    if stream is None:
        idx = device.index if device is not None and device.index is not None else torch.cuda.current_device()
        if _raw_stream is not None:
            return int(_raw_stream(idx))
        stream = torch.cuda.current_stream(idx)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None)
_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """Context in which `device` is current: entering it costs nothing when it
    already is (a kernel launches on the current device's stream)."""
    if _current_device is not None and _current_device() == device.index:
        return _HERE
    return torch.cuda.device(device)


_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _capturing(stream, device: torch.device) -> bool:
    """Whether a CUDA graph is being captured on the stream."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        return _is_capturing()


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """An output or workspace of a call on `stream` (None: the current one),
    allocated as that stream's memory: one of the current stream's could still
    be in use there by a tensor freed before, and could be handed out there
    again before the call has passed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class Rotation:
    """Owner of a paro_rot handle (device-resident prepared rotation)."""

    def __init__(self, pairs: np.ndarray, theta: np.ndarray, alpha: np.ndarray, group: int = 128):
        pairs = np.ascontiguousarray(pairs, dtype=np.int16)
        theta = np.ascontiguousarray(theta, dtype=np.float32)
        alpha = np.ascontiguousarray(alpha, dtype=np.float32)
        K = int(pairs.shape[0]) if pairs.ndim == 4 else 0
        P = int(pairs.shape[2]) if K else 0
        self.in_features = int(alpha.shape[0])
        self.K, self.P, self.group = K, P, int(group)
        h = _vp()
        _check("paro_rot_create", lib().paro_rot_create(
            ctypes.byref(h), self.in_features, group, K, P,
            pairs.ctypes.data if K else None, theta.ctypes.data if K else None, alpha.ctypes.data))
        self.handle = h

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            _check("paro_rot_destroy", lib().paro_rot_destroy(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def paro_rot_create(pairs, theta, alpha, group: int = 128) -> Rotation:
    return Rotation(pairs, theta, alpha, group)


def paro_rotate(rot: Rotation, X: torch.Tensor, Xr: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _dev(X, torch.float16, "X")
    if Xr is None:
        Xr = _empty(X.shape, torch.float16, X.device, stream)
    _dev(Xr, torch.float16, "Xr")
    if X.shape != Xr.shape or X.dim() != 2 or X.shape[1] != rot.in_features:
        raise ValueError("X/Xr must be [tokens][in_features]")
    _check("paro_rotate", lib().paro_rotate(rot.handle, X.data_ptr(), Xr.data_ptr(), X.shape[0], _stream(stream, X.device)))
    return Xr


def paro_fault_status(clear: bool = False) -> int:
    """0, or the code of a bounded in-kernel wait that ran out (synchronous)."""
    c = _int()
    _check("paro_fault_status", lib().paro_fault_status(ctypes.byref(c), 1 if clear else 0))
    return c.value


def paro_check_wait_timeout(limit_us: int = 1000, stream=None) -> None:
    """Enqueue the self-test kernel whose bounded wait runs out (code 6)."""
    _check("paro_check_wait_timeout", lib().paro_check_wait_timeout(int(limit_us), _stream(stream)))


def paro_pack_size(in_features: int, out_features: int, group: int = 128):
    q, s, z = _sz(), _sz(), _sz()
    if group == 128:
        _check("paro_pack_size", lib().paro_pack_size(in_features, out_features, ctypes.byref(q), ctypes.byref(s),
                                                      ctypes.byref(z)))
    else:
        _check("paro_pack_size_ex", lib().paro_pack_size_ex(in_features, out_features, group, ctypes.byref(q),
                                                            ctypes.byref(s), ctypes.byref(z)))
    return q.value, s.value, z.value


@functools.lru_cache(maxsize=None)
def _packed_bytes(in_features: int, rows: int, group: int):
    return paro_pack_size(in_features, rows, group)


def _weights(qw, sp, zp, in_features: int, rows: int, group: int, device: int):
    """Data pointers of packed weights, which must hold `rows` output rows of
    in_features channels in groups of `group` and lie on CUDA device `device`:
    the kernels read that much from there."""
    need = _packed_bytes(in_features, rows, group)
    for name, t, n in zip(("qweight", "scales", "zeros"), (qw, sp, zp), need):
        if isinstance(t, torch.Tensor) and t.dtype is torch.uint8 and t.get_device() == device >= 0 \
                and t.numel() >= n and t.is_contiguous():
            continue
        _dev(t, torch.uint8, name)                          # says what is wrong, if not the size or the place
        if t.numel() < n:
            raise ValueError(f"{name} holds {t.numel()} bytes, {n} needed for {rows} x {in_features} in groups of {group}")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, not on CUDA device {device}")
    return qw.data_ptr(), sp.data_ptr(), zp.data_ptr()


def _any(t, dtype, name) -> int:
    """Data pointer of a contiguous tensor on the device or on the host."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    return t.data_ptr()


def _logical(q, s, z, group: int, device: torch.device):
    """Data pointers of logical weights for a pack into memory of `device`,
    after checks of their sizes and that what is on a GPU is on that one."""
    ptrs = _any(q, torch.uint8, "q"), _any(s, torch.float16, "s"), _any(z, torch.uint8, "z")
    n = q.shape[0] * (q.shape[1] // group)
    if s.numel() != n or z.numel() != n:
        raise ValueError("s and z must be [out][in/group]")
    for name, t in (("q", q), ("s", s), ("z", z)):
        if t.is_cuda and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the packed weights on {device}")
    return ptrs


def paro_pack_weights(q: torch.Tensor, s: torch.Tensor, z: torch.Tensor, stream=None, device=None,
                      group: int = 128):
    """Logical (q uint8 [out][in], s fp16 [out][in/group], z uint8
    [out][in/group]), on the device or on the host -> device format
    (qweight, scales, zeros) as uint8 tensors on `device` (default: q's
    device, else the current one)."""
    out_f, in_f = q.shape
    sizes = paro_pack_size(in_f, out_f, group)
    dev = device or (q.device if q.is_cuda else torch.device("cuda", torch.cuda.current_device()))
    qw, sp, zp = (_empty(n, torch.uint8, dev, stream) for n in sizes)
    logical = _logical(q, s, z, group, qw.device)
    _check("paro_pack_weights_ex", lib().paro_pack_weights_ex(
        *logical, in_f, out_f, group, qw.data_ptr(), sp.data_ptr(), zp.data_ptr(), _stream(stream, qw.device)))
    return qw, sp, zp


def paro_dequant(qw, sp, zp, in_features: int, out_features: int, stream=None, group: int = 128) -> torch.Tensor:
    pq, ps, pz = _weights(qw, sp, zp, in_features, out_features, group, qw.get_device())
    W = _empty((out_features, in_features), torch.float16, qw.device, stream)
    _check("paro_dequant_ex", lib().paro_dequant_ex(pq, ps, pz, in_features, out_features, group, W.data_ptr(),
                                                    _stream(stream, qw.device)))
    return W


def paro_quantize_weights(rot: Rotation, W: torch.Tensor, stream=None):
    """W fp16 [out][in] -> (q uint8 [out][in], s fp16 [out][G], z uint8 [out][G]) of T W,
    G = in / the handle's group size."""
    out_f, in_f = W.shape
    G = in_f // rot.group
    w = _dev(W, torch.float16, "W")
    q = _empty((out_f, in_f), torch.uint8, W.device, stream)
    s = _empty((out_f, G), torch.float16, W.device, stream)
    z = _empty((out_f, G), torch.uint8, W.device, stream)
    _check("paro_quantize_weights", lib().paro_quantize_weights(
        rot.handle, w, out_f, q.data_ptr(), s.data_ptr(), z.data_ptr(), _stream(stream, W.device)))
    return q, s, z


def paro_linear_workspace_size(tokens: int, in_features: int, out_features: int) -> int:
    b = _sz()
    _check("paro_linear_workspace_size", lib().paro_linear_workspace_size(tokens, in_features, out_features, ctypes.byref(b)))
    return b.value


def workspace(tokens: int, in_features: int, out_features: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size paro_linear needs (allocated by torch)."""
    n = paro_linear_workspace_size(tokens, in_features, out_features)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def _scratch(tokens: int, in_features: int, out_features: int, device, stream) -> torch.Tensor:
    """A workspace for one call on `stream`, not filled."""
    n = paro_linear_workspace_size(tokens, in_features, out_features)
    return _empty(max(n, 16), torch.uint8, device, stream)


def paro_linear(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, out_features: int,
                Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    if Y is None:
        Y = _empty((T, out_features), torch.float16, X.device, stream)
    if ws is None:
        ws = _scratch(T, in_f, out_features, X.device, stream)
    _check("paro_linear", lib().paro_linear(
        rot.handle if rot is not None else None, x,
        *_weights(qw, sp, zp, in_f, out_features, 128, X.get_device()),
        _dev(Y, torch.float16, "Y"), T, in_f, out_features, _dev(ws, torch.uint8, "workspace"), ws.numel(),
        _stream(stream, X.device)))
    return Y


def paro_linear_bias(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, bias: Optional[torch.Tensor],
                     out_features: int, Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """paro_linear + bias (fp16 [out_features] CUDA tensor, or None)."""
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    if Y is None:
        Y = _empty((T, out_features), torch.float16, X.device, stream)
    if ws is None:
        ws = _scratch(T, in_f, out_features, X.device, stream)
    b = None
    if bias is not None:
        if bias.numel() != out_features:
            raise ValueError("bias must have out_features elements")
        b = _dev(bias, torch.float16, "bias")
    _check("paro_linear_bias", lib().paro_linear_bias(
        rot.handle if rot is not None else None, x,
        *_weights(qw, sp, zp, in_f, out_features, 128, X.get_device()), b,
        _dev(Y, torch.float16, "Y"), T, in_f, out_features, _dev(ws, torch.uint8, "workspace"), ws.numel(),
        _stream(stream, X.device)))
    return Y


def paro_rotate_once(X: torch.Tensor, pairs, theta, alpha, group: int = 128, stream=None) -> torch.Tensor:
    """X T^-1 from (pairs, theta, alpha) without a handle (allocating, synchronous)."""
    pairs = np.ascontiguousarray(pairs, dtype=np.int16)
    theta = np.ascontiguousarray(theta, dtype=np.float32)
    alpha = np.ascontiguousarray(alpha, dtype=np.float32)
    K = int(pairs.shape[0])
    P = int(pairs.shape[2]) if K else 0
    x = _dev(X, torch.float16, "X")
    Xr = _empty(X.shape, torch.float16, X.device, stream)
    T, in_f = X.shape
    _check("paro_rotate_once", lib().paro_rotate_once(
        x, Xr.data_ptr(), T, in_f, pairs.ctypes.data if K else None,
        theta.ctypes.data if K else None, alpha.ctypes.data, K, group, P, _stream(stream, X.device)))
    return Xr


def paro_linear_once(X: torch.Tensor, pairs, theta, alpha, qw, sp, zp, out_features: int,
                     stream=None) -> torch.Tensor:
    """Y = (X T^-1) w_hat^T from (pairs, theta, alpha) without a handle
    (allocating, synchronous)."""
    pairs = np.ascontiguousarray(pairs, dtype=np.int16)
    theta = np.ascontiguousarray(theta, dtype=np.float32)
    alpha = np.ascontiguousarray(alpha, dtype=np.float32)
    K = int(pairs.shape[0])
    P = int(pairs.shape[2]) if K else 0
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    Y = _empty((T, out_features), torch.float16, X.device, stream)
    _check("paro_linear_once", lib().paro_linear_once(
        x, pairs.ctypes.data if K else None, theta.ctypes.data if K else None,
        alpha.ctypes.data, *_weights(qw, sp, zp, in_f, out_features, 128, X.get_device()),
        _dev(Y, torch.float16, "Y"), T, in_f, out_features, K, P,
        _stream(stream, X.device)))
    return Y


def paro_linear_ex(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, out_features: int, group: int = 128,
                   bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The layer with weights quantised in groups of `group` channels (128 or 64)."""
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    if Y is None:
        Y = _empty((T, out_features), torch.float16, X.device, stream)
    if ws is None:
        ws = _scratch(T, in_f, out_features, X.device, stream)
    b = None
    if bias is not None:
        if bias.numel() != out_features:
            raise ValueError("bias must have out_features elements")
        b = _dev(bias, torch.float16, "bias")
    _check("paro_linear_ex", lib().paro_linear_ex(
        rot.handle if rot is not None else None, x,
        *_weights(qw, sp, zp, in_f, out_features, group, X.get_device()), b, group,
        _dev(Y, torch.float16, "Y"), T, in_f, out_features, _dev(ws, torch.uint8, "workspace"), ws.numel(),
        _stream(stream, X.device)))
    return Y


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _bias(bias: Optional[torch.Tensor], n: int) -> Optional[int]:
    if bias is None:
        return None
    if bias.numel() != n:
        raise ValueError(f"bias must have {n} elements")
    return _dev(bias, torch.float16, "bias")


def _same_device(X: torch.Tensor, **others) -> None:
    for name, t in others.items():
        if t is not None and t.device != X.device:
            raise ValueError(f"{name} is on {t.device}, not on {X.device}")


def paro_linear_act(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, out_features: int, act: str = "none",
                    group: int = 128, bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                    Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = act((X T^-1) w_hat^T + bias) + residual, rounded once; Y may be the residual."""
    a, b = _act(act), _bias(bias, out_features)
    x = _dev(X, torch.float16, "X")
    _same_device(X, bias=bias, workspace=ws)
    T, in_f = X.shape
    w = _weights(qw, sp, zp, in_f, out_features, group, X.get_device())
    shape = (T, out_features)
    r = None if residual is None else _f16(residual, shape, X.get_device(), "residual")
    Y = _out(Y, shape, torch.float16, X.device, "Y", stream)
    if ws is None:
        ws = _scratch(T, in_f, out_features, X.device, stream)
    with _on(X.device):
        _check("paro_linear_act", lib().paro_linear_act(
            rot.handle if rot is not None else None, x, *w, b, r, a, group, Y.data_ptr(), T, in_f, out_features,
            _dev(ws, torch.uint8, "workspace"), ws.numel(), _stream(stream, X.device)))
    return Y


def paro_pack_gated(q: torch.Tensor, s: torch.Tensor, z: torch.Tensor, stream=None, device=None, group: int = 128):
    """Logical gate rows, then up rows (q uint8 [2 inter][in], s fp16 and z uint8
    [2 inter][in/group]), on the device or on the host -> the device format of
    paro_linear_gated (qweight, scales, zeros)."""
    out_f, in_f = q.shape
    if out_f % 2:
        raise ValueError("q must hold as many up rows as gate rows")
    if group > 0 and (s.shape != (out_f, in_f // group) or z.shape != s.shape):
        raise ValueError("s and z must be [2 inter][in/group]")
    sizes = paro_pack_size(in_f, out_f, group)
    dev = device or (q.device if q.is_cuda else torch.device("cuda", torch.cuda.current_device()))
    qw, sp, zp = (_empty(n, torch.uint8, dev, stream) for n in sizes)
    logical = _logical(q, s, z, group, qw.device)
    with _on(qw.device):
        _check("paro_pack_gated", lib().paro_pack_gated(
            *logical, in_f, out_f // 2, group, qw.data_ptr(), sp.data_ptr(), zp.data_ptr(), _stream(stream, qw.device)))
    return qw, sp, zp


def paro_linear_gated(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, inter_features: int, act: str = "silu",
                      group: int = 128, bias: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """H = act((X T^-1) w_gate^T + b_gate) * ((X T^-1) w_up^T + b_up), weights
    from paro_pack_gated, bias [2 inter] (the gate's first)."""
    a, b = _act(act), _bias(bias, 2 * inter_features)
    x = _dev(X, torch.float16, "X")
    _same_device(X, bias=bias, workspace=ws)
    T, in_f = X.shape
    w = _weights(qw, sp, zp, in_f, 2 * inter_features, group, X.get_device())
    H = _out(H, (T, inter_features), torch.float16, X.device, "H", stream)
    if ws is None:
        ws = _scratch(T, in_f, 2 * inter_features, X.device, stream)
    with _on(X.device):
        _check("paro_linear_gated", lib().paro_linear_gated(
            rot.handle if rot is not None else None, x, *w, b, a, group, H.data_ptr(), T, in_f, inter_features,
            _dev(ws, torch.uint8, "workspace"), ws.numel(), _stream(stream, X.device)))
    return H


class ParoLinear:
    """A prepared layer for repeated calls (a decode loop): the rotation
    handle, the packed weights, the bias and a workspace are checked once
    here; a call checks only X, Y and the residual and hands raw pointers to
    the same C entry points as paro_linear_ex and paro_linear_act (the latter
    with an activation or a residual). The workspace is owned by the object
    and has the size of the largest batch seen; an outgrown one is kept if it
    may still be used, by a CUDA graph that captured a call or by a call on
    another stream than the one whose memory it is. So calls on one object must
    not overlap on the GPU (one stream, or events), as for paro_linear's
    workspace, and the object must outlive the graphs that captured it and its
    calls on other streams. The object keeps references to the tensors it was
    given."""

    _width_factor = 1                                   # rows of the weights per output column

    def __init__(self, rot: Optional[Rotation], qw, sp, zp, in_features: int, out_features: int, group: int = 128,
                 bias: Optional[torch.Tensor] = None, device=None, act: str = "none"):
        if rot is not None and (rot.group != group or rot.in_features != in_features):
            raise ValueError("the rotation was prepared for another group size or input width")
        self.rot, self.in_features, self.out_features, self.group = rot, int(in_features), int(out_features), group
        self.act = act
        self._a = _act(act)
        self._tensors = (qw, sp, zp, bias)                 # kept alive for the pointers below
        self._h = rot.handle if rot is not None else None
        rows = self._width_factor * self.out_features
        _dev(qw, torch.uint8, "qweight")
        self._index = qw.get_device()
        self._qw, self._sp, self._zp = _weights(qw, sp, zp, self.in_features, rows, group, self._index)
        self._b = _bias(bias, rows)
        _same_device(qw, bias=bias)
        self.device = qw.device
        if device is not None and torch.empty(0, device=device).device != self.device:
            raise ValueError(f"the layer is on {self.device}, where its weights are, not on {device}")
        self._ws = None
        self._ws_tokens = 0
        self._ws_stream = None                             # raw stream whose memory the workspace is
        self._ws_shared = False                            # a graph or another stream may use it
        self._kept = []                                    # outgrown workspaces that were shared
        self._f = lib().paro_linear_ex
        self._f_act = lib().paro_linear_act

    def _workspace(self, T: int, stream=None) -> None:
        if T > self._ws_tokens or self._ws is None:
            if self._ws_shared:
                self._kept.append(self._ws)
            self._ws = None                                # its memory may serve the next one
            self._ws = _scratch(T, self.in_features, self._width_factor * self.out_features, self.device, stream)
            self._ws_tokens, self._ws_stream, self._ws_shared = T, _stream(stream, self.device), False

    def _prepare(self, X, Y, stream):
        """(tokens, Y, raw stream) of a call, after its checks."""
        T = X.shape[0]
        if not X.is_cuda or X.dtype is not torch.float16 or not X.is_contiguous() or X.dim() != 2 \
                or X.shape[1] != self.in_features:
            raise TypeError(f"X must be a contiguous fp16 CUDA tensor [tokens][{self.in_features}]")
        if Y is None:
            Y = _empty((T, self.out_features), torch.float16, X.device, stream)
        elif not Y.is_cuda or Y.dtype is not torch.float16 or not Y.is_contiguous() or Y.numel() != T * self.out_features:
            raise TypeError(f"Y must be a contiguous fp16 CUDA tensor [tokens][{self.out_features}]")
        if X.get_device() != Y.get_device() or X.get_device() != self._index:
            raise ValueError(f"X on {X.device}, Y on {Y.device}, the layer on {self.device}")
        if T > self._ws_tokens or self._ws is None:
            self._workspace(T, stream)
        if stream is None and _raw_stream is not None:
            raw = int(_raw_stream(X.get_device()))
        else:
            raw = _stream(stream, X.device)
        # (the default stream, raw 0, cannot be captured; asking costs 0.3 us)
        if not self._ws_shared and (raw != self._ws_stream or raw != 0 and
                                    (_is_capturing() if stream is None else _capturing(stream, X.device))):
            self._ws_shared = True
        return T, Y, raw

    def __call__(self, X: torch.Tensor, Y: Optional[torch.Tensor] = None, stream=None,
                 residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        T, Y, sp = self._prepare(X, Y, stream)
        if _current_device is not None and _current_device() != self._index:   # launch on the layer's device
            with torch.cuda.device(self._index):
                return self(X, Y, sp, residual)
        if residual is None and self._a == 0:
            st = self._f(self._h, X.data_ptr(), self._qw, self._sp, self._zp, self._b, self.group, Y.data_ptr(), T,
                         self.in_features, self.out_features, self._ws.data_ptr(), self._ws.numel(), sp)
            if st != PARO_OK:
                _check("paro_linear_ex", st)
            return Y
        r = None if residual is None else _f16(residual, (T, self.out_features), X.get_device(), "residual")
        st = self._f_act(self._h, X.data_ptr(), self._qw, self._sp, self._zp, self._b, r, self._a, self.group,
                         Y.data_ptr(), T, self.in_features, self.out_features, self._ws.data_ptr(), self._ws.numel(), sp)
        if st != PARO_OK:
            _check("paro_linear_act", st)
        return Y


class ParoGated(ParoLinear):
    """The prepared form of paro_linear_gated: weights from paro_pack_gated,
    bias [2 inter_features]; a call returns H [tokens][inter_features]."""

    _width_factor = 2

    def __init__(self, rot: Optional[Rotation], qw, sp, zp, in_features: int, inter_features: int, group: int = 128,
                 bias: Optional[torch.Tensor] = None, device=None, act: str = "silu"):
        super().__init__(rot, qw, sp, zp, in_features, inter_features, group, bias, device, act)
        self.inter_features = self.out_features
        self._f_gated = lib().paro_linear_gated

    def __call__(self, X: torch.Tensor, H: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T, H, sp = self._prepare(X, H, stream)
        if _current_device is not None and _current_device() != self._index:   # launch on the layer's device
            with torch.cuda.device(self._index):
                return self(X, H, sp)
        st = self._f_gated(self._h, X.data_ptr(), self._qw, self._sp, self._zp, self._b, self._a, self.group,
                           H.data_ptr(), T, self.in_features, self.out_features, self._ws.data_ptr(), self._ws.numel(), sp)
        if st != PARO_OK:
            _check("paro_linear_gated", st)
        return H


def paro_linear_partial(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, out_features: int, group: int = 128,
                        Yf: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """A row-parallel rank's unrounded fp32 share of Y over its input slice."""
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    if Yf is None:
        Yf = _empty((T, out_features), torch.float32, X.device, stream)
    if ws is None:
        ws = _scratch(T, in_f, out_features, X.device, stream)
    _check("paro_linear_partial", lib().paro_linear_partial(
        rot.handle if rot is not None else None, x,
        *_weights(qw, sp, zp, in_f, out_features, group, X.get_device()), group,
        _dev(Yf, torch.float32, "Yf"), T, in_f, out_features, _dev(ws, torch.uint8, "workspace"), ws.numel(),
        _stream(stream, X.device)))
    return Yf


def paro_finalize(Yf: torch.Tensor, bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """fp16(Yf + bias), one rounding."""
    yf = _dev(Yf, torch.float32, "Yf")
    T, out_f = Yf.shape
    if Y is None:
        Y = _empty((T, out_f), torch.float16, Yf.device, stream)
    b = _dev(bias, torch.float16, "bias") if bias is not None else None
    _check("paro_finalize", lib().paro_finalize(yf, b, _dev(Y, torch.float16, "Y"), T, out_f,
                                                _stream(stream, Yf.device)))
    return Y


def paro_linear_noalloc(rot: Optional[Rotation], X: torch.Tensor, qw, sp, zp, out_features: int,
                        Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode (tokens <= 16) with the library's static scratch: no workspace,
    no device allocation inside the call (Y is allocated here only if not given)."""
    x = _dev(X, torch.float16, "X")
    T, in_f = X.shape
    if Y is None:
        Y = _empty((T, out_features), torch.float16, X.device, stream)
    _check("paro_linear_noalloc", lib().paro_linear_noalloc(
        rot.handle if rot is not None else None, x,
        *_weights(qw, sp, zp, in_f, out_features, 128, X.get_device()),
        _dev(Y, torch.float16, "Y"), T, in_f, out_features, _stream(stream, X.device)))
    return Y


def _f16(t: torch.Tensor, shape, device: int, name: str, dtype: torch.dtype = torch.float16) -> int:
    """Data pointer of a contiguous fp16 (or `dtype`) tensor of this shape on CUDA device `device`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _dev(t, dtype, name)                                    # says what is wrong, if not the place or the shape
    raise ValueError(f"{name} must be {list(shape)} on cuda:{device}, got {list(t.shape)} on {t.device}")


def _launch(fn, device: int, stream, *args) -> int:
    """fn(*args, raw stream) with `device` current, on the given stream or
    that device's current one."""
    if _current_device is None or _current_device() != device:
        with torch.cuda.device(device):
            return fn(*args, _stream(stream, torch.device("cuda", device)))
    if stream is None and _raw_stream is not None:
        return fn(*args, _raw_stream(device))
    return fn(*args, _stream(stream, torch.device("cuda", device)))


def _norm_args(X, weight, residual, bias, H, stream):
    """Shape, pointers and H of a norm after the checks its two forms share; H
    is allocated when a residual, a bias or fp32 sums make it differ from X."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2 or X.dtype not in (torch.float16, torch.float32):
        raise TypeError("X must be a [tokens][features] fp16 or fp32 CUDA tensor")
    x32 = X.dtype is torch.float32
    shape, dev = X.shape, X.get_device()
    x = _dev(X, X.dtype, "X")
    row = shape[1:]
    if H is None and (residual is not None or bias is not None or x32):
        H = _empty(shape, torch.float16, X.device, stream)
    return shape, (x, int(x32),
                   None if residual is None else _f16(residual, shape, dev, "residual"),
                   None if bias is None else _f16(bias, row, dev, "bias"),
                   _f16(weight, row, dev, "weight")), \
        None if H is None else _f16(H, shape, dev, "H"), H


def _out(t, shape, dtype, device, name, stream):
    """An output: allocated, or the given tensor after its checks."""
    if t is None:
        return _empty(shape, dtype, device, stream)
    _dev(t, dtype, name)
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {list(shape)} on {device}, got {list(t.shape)} on {t.device}")
    return t


def paro_rmsnorm(X: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None,
                 Y: Optional[torch.Tensor] = None, stream=None):
    """(Y, H): v = X + bias + residual, H = fp16(v), Y = fp16 of v's
    root-mean-square norm times weight. X fp16, or fp32 sums of a row-parallel
    layer. H is None when nothing is added to an fp16 X and no H is given;
    H=residual updates the residual stream in place."""
    shape, args, h, H = _norm_args(X, weight, residual, bias, H, stream)
    if Y is None:
        Y = _empty(shape, torch.float16, X.device, stream)
    dev = X.get_device()
    st = _launch(lib().paro_rmsnorm, dev, stream, *args, eps, h, _f16(Y, shape, dev, "Y"), *shape)
    if st != PARO_OK:
        _check("paro_rmsnorm", st)
    return Y, H


def paro_rmsnorm_q8(X: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                    bias: Optional[torch.Tensor] = None, scale_group: int = 128, H: Optional[torch.Tensor] = None,
                    Y: Optional[torch.Tensor] = None, S: Optional[torch.Tensor] = None, stream=None):
    """(codes, scales, H): paro_rmsnorm with Y as float8_e4m3fn codes and fp32
    scales [tokens][ceil(features / 128)] (scale_group 128) or [tokens][1]
    (scale_group 0: one scale per row)."""
    shape, args, h, H = _norm_args(X, weight, residual, bias, H, stream)
    T, F = shape
    scales, dev = (T, -(-F // 128) if scale_group else 1), X.get_device()
    if Y is None:
        Y = _empty(shape, torch.float8_e4m3fn, X.device, stream)
    if S is None:
        S = _empty(scales, torch.float32, X.device, stream)
    st = _launch(lib().paro_rmsnorm_q8, dev, stream, *args, eps, scale_group, h,
                 _f16(Y, shape, dev, "Y", torch.float8_e4m3fn), _f16(S, scales, dev, "S", torch.float32), T, F)
    if st != PARO_OK:
        _check("paro_rmsnorm_q8", st)
    return Y, S, H


def paro_q8_expand(Q: torch.Tensor, S: torch.Tensor, scale_group: int = 128, Y: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """fp16(code * scale) of paro_rmsnorm_q8's codes and scales."""
    q, s = _dev(Q, torch.float8_e4m3fn, "Q"), _dev(S, torch.float32, "S")
    if Q.dim() != 2 or S.shape != (Q.shape[0], -(-Q.shape[1] // 128) if scale_group else 1) or S.device != Q.device:
        raise ValueError("S must hold one scale per row, or per 128 channels of a row, of Q [tokens][features]")
    T, F = Q.shape
    Y = _out(Y, (T, F), torch.float16, Q.device, "Y", stream)
    with _on(Q.device):
        _check("paro_q8_expand", lib().paro_q8_expand(q, s, scale_group, Y.data_ptr(), T, F,
                                                      _stream(stream, Q.device)))
    return Y
