"""Binding of the layer norm (``include/swiglu_norm.h``), forward and backward.

Argument marshalling only, like the rest of the package.

    y, mean, rstd = swiglu_layer_norm_fwd(x, w, b, eps, return_stats=True)
    dx, dw, db = swiglu_layer_norm_bwd(dy, x, mean, rstd, w)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import SwigluError, _DTYPE, lib
from .moe import _F32, _call, _current_device, _float_type, _given, _ptr, _rows, _weights

# every symbol include/swiglu_norm.h declares
NORM_EXPORTS = ("swiglu_layer_norm_fwd", "swiglu_layer_norm_bwd_workspace_size", "swiglu_layer_norm_bwd",
                "swiglu_layer_norm_timeout_flag")


def _declare() -> None:
    i64, vp, i32, size = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for name, args in (
            ("swiglu_layer_norm_fwd", [vp] * 6 + [i64] * 4 + [ctypes.c_float, i32, i32, vp]),
            ("swiglu_layer_norm_bwd_workspace_size", [i64, i64, i32, ctypes.POINTER(size)]),
            ("swiglu_layer_norm_bwd", [vp] * 9 + [size] + [i64] * 5 + [i32, i32, vp]),
            ("swiglu_layer_norm_timeout_flag", [ctypes.POINTER(ctypes.c_int)])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i32


_declare()


def _matrix(x: torch.Tensor, name: str):
    """(rows, row stride, n) of a [..., n] tensor."""
    if x.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    n = x.shape[-1]
    if n:
        return (*_rows(x, n, name), n)
    rows = 1
    for d in x.shape[:-1]:
        rows *= d
    return rows, 0, 0


def _row_stride(t: torch.Tensor, x: torch.Tensor, rows: int, n: int, name: str) -> int:
    """The row stride of a tensor the caller gave, checked to hold rows like x's."""
    if t.shape == x.shape and t.dtype is x.dtype and t.is_contiguous() and t.get_device() == x.get_device():
        return n
    return _given(t, rows, n, x.dtype, x.device, name) if n else 0


# Results are allocated by torch's public call alone, so that dispatch modes, profilers and the
# deterministic fill of uninitialised memory see them: no way past the dispatcher is taken,
# though one would save some 1.5 us of a call.
_empty_cuda = None


def _empty(shape, dtype: torch.dtype, like: torch.Tensor) -> torch.Tensor:
    """An empty contiguous tensor on like's (CUDA) device."""
    return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(need: int, x: torch.Tensor, stream) -> torch.Tensor:
    """A workspace that goes back to the allocator as memory of the stream that uses it."""
    if stream is None:
        return _empty((need,), torch.uint8, x)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=x.device)


def _param(t: torch.Tensor, x: torch.Tensor, n: int, dtype, name: str) -> torch.dtype:
    """The dtype of a parameter or its gradient: x's or float32, and ``dtype`` if that is
    not None."""
    if t.get_device() != x.get_device():
        raise ValueError("all tensors must be on the same CUDA device")
    own = t.dtype
    if (own is not x.dtype and own is not _F32) or (dtype is not None and own is not dtype):
        raise ValueError(f"weight, bias and their gradients must all be {x.dtype} or all float32")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements")
    return own


def swiglu_layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor = None, bias: torch.Tensor = None, eps: float = 1e-5,
                          y: torch.Tensor = None, mean: torch.Tensor = None, rstd: torch.Tensor = None,
                          return_stats: bool = False, stream=None):
    """y = (x - mean) rstd weight + bias over the last dimension of x [..., n];
    ``weight`` and ``bias`` [n] (x's dtype or float32) are optional.  With
    ``return_stats`` (y, mean, rstd): the float32 statistics of the rows, shaped as
    x without its last dimension, which the backward takes."""
    code = _float_type(x)
    rows, sx, n = _matrix(x, "x")
    shape, device = x.shape, x.device
    dtype = None
    if weight is not None:
        dtype = _param(weight, x, n, None, "weight")
    if bias is not None:
        dtype = _param(bias, x, n, dtype, "bias")
    sy = n
    if y is None:
        y = _empty(shape, x.dtype, x)
    else:
        sy = _row_stride(y, x, rows, n, "y")
    if return_stats:
        lead = shape[:-1]
        if mean is None:
            mean = _empty(lead, _F32, x)
        if rstd is None:
            rstd = _empty(lead, _F32, x)
    _call("swiglu_layer_norm_fwd", lib.swiglu_layer_norm_fwd, x, stream, x.data_ptr(), _ptr(weight), _ptr(bias),
          y.data_ptr(), None if mean is None else _weights(mean, rows, device, "mean"),
          None if rstd is None else _weights(rstd, rows, device, "rstd"), rows, n, sx, sy, eps, code,
          code if dtype is None else _DTYPE[dtype])
    return (y, mean, rstd) if return_stats else y


def layer_norm_bwd_workspace_bytes(rows: int, n: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace of the backward on the current device."""
    if dtype not in _DTYPE:
        raise ValueError("dtype must be float32 or bfloat16")
    return _workspace_bytes(rows, n, _DTYPE[dtype], _current_device())


@functools.lru_cache(maxsize=1024)  # a device's answer follows from the sizes
def _workspace_bytes(rows: int, n: int, code: int, device: int) -> int:
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        st = lib.swiglu_layer_norm_bwd_workspace_size(rows, n, code, ctypes.byref(out))
    if st != 0:
        raise SwigluError(st, "swiglu_layer_norm_bwd_workspace_size")
    return int(out.value)


def swiglu_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                          weight: torch.Tensor = None, bias_grad: bool = True, dx: torch.Tensor = None,
                          dweight: torch.Tensor = None, dbias: torch.Tensor = None, workspace: torch.Tensor = None,
                          stream=None, weight_grad: bool = True):
    """(dx, dweight, dbias) of the layer norm at x with the forward's mean and rstd.
    dweight is None without ``weight`` (or with ``weight_grad=False`` and no ``dweight``
    given), dbias without ``bias_grad`` (or a ``dbias`` given); both have the parameters'
    dtype (x's without ``weight``)."""
    code = _float_type(x)
    rows, sx, n = _matrix(x, "x")
    device = x.device
    sdy = _row_stride(dy, x, rows, n, "dy")
    if weight is None and dweight is not None:
        raise ValueError("dweight is the gradient of weight: it needs weight")
    dtype = None
    if weight is not None:
        dtype = _param(weight, x, n, None, "weight")
        if dweight is not None:
            _param(dweight, x, n, dtype, "dweight")
        elif weight_grad:
            dweight = _empty(weight.shape, dtype, x)
    if dbias is not None:
        dtype = _param(dbias, x, n, dtype, "dbias")
    elif bias_grad:
        dbias = _empty((n,), x.dtype if dtype is None else dtype, x)
    sdx = n
    if dx is None:
        dx = _empty(x.shape, x.dtype, x)
    else:
        sdx = _row_stride(dx, x, rows, n, "dx")
    need = _workspace_bytes(rows, n, code, x.get_device())
    if workspace is None:
        workspace = _scratch(need, x, stream) if need else None
    elif workspace.device != device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {device}")
    _call("swiglu_layer_norm_bwd", lib.swiglu_layer_norm_bwd, x, stream, dy.data_ptr(), x.data_ptr(),
          _weights(mean, rows, device, "mean"), _weights(rstd, rows, device, "rstd"), _ptr(weight), dx.data_ptr(),
          _ptr(dweight), _ptr(dbias), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), rows, n, sdy, sx, sdx, code,
          code if dtype is None else _DTYPE[dtype])
    return dx, dweight, dbias


def layer_norm_timeout_flag() -> int:
    """1 if any layer norm so far gave up on an internal wait, else 0 (synchronises with
    the current device)."""
    out = ctypes.c_int(0)
    st = lib.swiglu_layer_norm_timeout_flag(ctypes.byref(out))
    if st != 0:
        raise SwigluError(st, "swiglu_layer_norm_timeout_flag")
    return int(out.value)


__all__ = ["swiglu_layer_norm_fwd", "swiglu_layer_norm_bwd", "layer_norm_bwd_workspace_bytes",
           "layer_norm_timeout_flag", "NORM_EXPORTS"]
