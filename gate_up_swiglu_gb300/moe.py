"""Binding of the routed experts' operators (``include/swiglu_moe.h``): the
grouped matrix products and the 8-bit activation checkpoint.

Argument marshalling only, like the rest of the package.  Rows are sorted by
expert and ``ends`` is a CUDA int32 tensor, the running sum of the rows per
expert; rows from ``ends[-1]`` on belong to no expert, and their outputs are
zero.

    ends = counts.cumsum(0, dtype=torch.int32)               # [E]
    y, q, s = swiglu_grouped_fc1_fwd(x, w1, ends, probs, save="fp8")
    out = swiglu_grouped_mm_fwd(y, w2, ends)
    ...
    dy = swiglu_grouped_mm_dgrad(dout, w2, ends)
    dfc1, dprobs, y = swiglu_ckpt8_bwd(dy, q, s, probs, return_y=True)
    dw2 = swiglu_grouped_mm_wgrad(dout, y, ends)

The checkpoint (``q``: torch.float8_e4m3fn, ``scales``: torch.float8_e8m0fnu)
holds each half of a row in blocks of 32 columns, one power of two per block.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_DTYPE, SWIGLU_BF16, SwigluError, _check_cuda, _on_device, _rows_view, _stream_handle,
               _vector, lib)

CKPT8_BLOCK = 32
MAX_GROUPS = 1024
Q_DTYPE = torch.float8_e4m3fn
SCALE_DTYPE = torch.float8_e8m0fnu

# every symbol include/swiglu_moe.h declares
MOE_EXPORTS = ("swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_grouped_fc1_fwd", "swiglu_grouped_mm_fwd",
               "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "swiglu_grouped_timeout_flag")


def _declare() -> None:
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name, args in (
            ("swiglu_ckpt8_fwd", [vp] * 5 + [i64] * 6 + [i32, vp]),
            ("swiglu_ckpt8_bwd", [vp] * 7 + [i64] * 7 + [i32, vp]),
            ("swiglu_grouped_fc1_fwd", [vp] * 8 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_fwd", [vp] * 4 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_dgrad", [vp] * 4 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_wgrad", [vp] * 4 + [i64] * 4 + [i32, i32, i32, vp]),
            ("swiglu_grouped_timeout_flag", [ctypes.POINTER(ctypes.c_int)])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i32


_declare()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name: str, t: torch.Tensor, stream, *args) -> None:
    with _on_device(t.device):
        st = getattr(lib, name)(*args, _stream_handle(t, stream))
    if st != 0:
        raise SwigluError(st, name)


def _same_device(t: torch.Tensor, *others) -> None:
    for o in others:
        if o is not None and o.device != t.device:
            raise ValueError("all tensors must be on the same CUDA device")


def _ckpt8_views(q, scales, rows, n):
    """Row strides of the codes and scales of a checkpoint of [rows, 2n]."""
    nb = -(-n // CKPT8_BLOCK)
    if q.dtype != Q_DTYPE or scales.dtype != SCALE_DTYPE:
        raise ValueError("a checkpoint is q (float8_e4m3fn) and scales (float8_e8m0fnu)")
    qrows, qcols, sq = _rows_view(q, "q")
    srows, scols, ss = _rows_view(scales, "scales")
    if (qrows, qcols) != (rows, 2 * n) or (srows, scols) != (rows, 2 * nb):
        raise ValueError(f"the checkpoint of [{rows}, {2 * n}] is q [{rows}, {2 * n}] and scales [{rows}, {2 * nb}]")
    return sq, ss


def swiglu_ckpt8_fwd(x: torch.Tensor, w: torch.Tensor = None, y: torch.Tensor = None, q: torch.Tensor = None,
                     scales: torch.Tensor = None, stream=None):
    """(y, q, scales): y = w[row] * silu(gate) * up and the 8-bit checkpoint of x.

    ``w`` (fp32, one weight per row of x) is optional."""
    if x.shape[-1] % 2:
        raise ValueError("x's last dimension must be even (gate and up halves)")
    lead, n = x.shape[:-1], x.shape[-1] // 2
    if y is None:
        y = torch.empty((*lead, n), dtype=x.dtype, device=x.device)
    if q is None:
        q = torch.empty((*lead, 2 * n), dtype=Q_DTYPE, device=x.device)
    if scales is None:
        scales = torch.empty((*lead, 2 * -(-n // CKPT8_BLOCK)), dtype=SCALE_DTYPE, device=x.device)
    _check_cuda(x, y)
    _same_device(x, w, q, scales)
    rows, _, sx = _rows_view(x, "x")
    yrows, yn, sy = _rows_view(y, "y")
    if (yrows, yn) != (rows, n):
        raise ValueError("y must be [..., n] with the rows of x")
    sq, ss = _ckpt8_views(q, scales, rows, n)
    if w is not None:
        _vector(w, "w", rows, torch.float32)
    _call("swiglu_ckpt8_fwd", x, stream, x.data_ptr(), _ptr(w), y.data_ptr(), q.data_ptr(), scales.data_ptr(), rows,
          n, sx, sy, sq, ss, _DTYPE[x.dtype])
    return y, q, scales


def swiglu_ckpt8_bwd(dy: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, w: torch.Tensor = None,
                     dx: torch.Tensor = None, dw: torch.Tensor = None, y: torch.Tensor = None,
                     return_y: bool = False, stream=None):
    """(dx, dw, y) of the SwiGLU at the checkpointed x: the input gradient, the
    fp32 gradient of the row weights (None without ``w``) and, with ``return_y``
    (or a ``y`` given), the forward's output made again from the checkpoint
    (else None)."""
    lead, n = dy.shape[:-1], dy.shape[-1]
    if dx is None:
        dx = torch.empty((*lead, 2 * n), dtype=dy.dtype, device=dy.device)
    if return_y and y is None:
        y = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    if w is not None and dw is None:
        dw = torch.empty(w.shape, dtype=torch.float32, device=dy.device)
    if w is None and dw is not None:
        raise ValueError("dw is the gradient of w: it needs w")
    _check_cuda(dy, dx, *([y] if y is not None else []))
    _same_device(dy, w, dw, q, scales)
    rows, _, sdy = _rows_view(dy, "dy")
    dxrows, dxcols, sdx = _rows_view(dx, "dx")
    if (dxrows, dxcols) != (rows, 2 * n):
        raise ValueError("dx must be [..., 2n] with the rows of dy")
    sy = 0
    if y is not None:
        yrows, yn, sy = _rows_view(y, "y")
        if (yrows, yn) != (rows, n):
            raise ValueError("y must have the shape of dy")
    sq, ss = _ckpt8_views(q, scales, rows, n)
    if w is not None:
        _vector(w, "w", rows, torch.float32)
        _vector(dw, "dw", rows, torch.float32)
    _call("swiglu_ckpt8_bwd", dy, stream, dy.data_ptr(), q.data_ptr(), scales.data_ptr(), _ptr(w), dx.data_ptr(),
          _ptr(dw), _ptr(y), rows, n, sdy, sq, ss, sdx, sy, _DTYPE[dy.dtype])
    return dx, dw, y


def _experts(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, cols: int, what: str):
    """Checks shared by the products: bf16 x [rows, *] and w [E, N, K], ends [E]."""
    _check_cuda(x, w)
    if x.dtype != torch.bfloat16:
        raise ValueError("the grouped products take bfloat16 tensors")
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError(f"{what} must be [rows, {cols}] and w [experts, N, K]")
    _ends(ends, x, w.shape[0])


def _ends(ends: torch.Tensor, x: torch.Tensor, groups: int) -> None:
    _vector(ends, "ends", groups, torch.int32)
    _same_device(x, ends)


def _contiguous(*ts) -> None:
    if not all(t is None or t.is_contiguous() for t in ts):
        raise ValueError("the grouped products need contiguous tensors")


def _result(t, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {like.device}")
    return t


def swiglu_grouped_fc1_fwd(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, probs: torch.Tensor = None,
                           y: torch.Tensor = None, save: str = None, fc1: torch.Tensor = None,
                           q: torch.Tensor = None, scales: torch.Tensor = None, stream=None):
    """The experts' first product with its activation: y[t] = probs[t] *
    silu(W[e] gate rows . x[t]) * (W[e] up rows . x[t]); x [rows, K], w [E, 2n, K]
    (gate rows first), probs (fp32, one per row) optional.

    ``save`` picks what the backward needs: None returns y; ``"bf16"`` (y, fc1)
    with the [rows, 2n] product rounded to bf16; ``"fp8"`` (y, q, scales) with its
    8-bit checkpoint."""
    if save not in (None, "bf16", "fp8"):
        raise ValueError('save must be None, "bf16" or "fp8"')
    _experts(x, w, ends, w.shape[-1], "x")
    (rows, K), (E, two_n, wk) = x.shape, w.shape
    if wk != K or two_n % 2:
        raise ValueError("w must be [experts, 2n, K] with x's K")
    n = two_n // 2
    nb = -(-n // CKPT8_BLOCK)
    y = _result(y, (rows, n), x.dtype, x, "y")
    fc1 = _result(fc1, (rows, two_n), x.dtype, x, "fc1") if save == "bf16" else None
    q = _result(q, (rows, two_n), Q_DTYPE, x, "q") if save == "fp8" else None
    scales = _result(scales, (rows, 2 * nb), SCALE_DTYPE, x, "scales") if save == "fp8" else None
    _contiguous(x, w, y, fc1, q, scales)
    if probs is not None:
        _vector(probs, "probs", rows, torch.float32)
        _same_device(x, probs)
    _call("swiglu_grouped_fc1_fwd", x, stream, x.data_ptr(), w.data_ptr(), ends.data_ptr(), _ptr(probs), y.data_ptr(),
          _ptr(fc1), _ptr(q), _ptr(scales), rows, E, n, K, SWIGLU_BF16)
    return (y, fc1) if save == "bf16" else (y, q, scales) if save == "fp8" else y


def swiglu_grouped_mm_fwd(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, y: torch.Tensor = None,
                          stream=None) -> torch.Tensor:
    """y[t] = W[e] x[t]: x [rows, K], w [E, N, K] -> y [rows, N]."""
    _experts(x, w, ends, w.shape[-1], "x")
    (rows, K), (E, N, wk) = x.shape, w.shape
    if wk != K:
        raise ValueError("w must be [experts, N, K] with x's K")
    y = _result(y, (rows, N), x.dtype, x, "y")
    _contiguous(x, w, y)
    _call("swiglu_grouped_mm_fwd", x, stream, x.data_ptr(), w.data_ptr(), ends.data_ptr(), y.data_ptr(), rows, E, N, K,
          SWIGLU_BF16)
    return y


def swiglu_grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, dx: torch.Tensor = None,
                            stream=None) -> torch.Tensor:
    """dx[t] = W[e]^T dy[t]: dy [rows, N], w [E, N, K] -> dx [rows, K]."""
    _experts(dy, w, ends, w.shape[1] if w.dim() == 3 else 0, "dy")
    (rows, N), (E, wn, K) = dy.shape, w.shape
    if wn != N:
        raise ValueError("w must be [experts, N, K] with dy's N")
    dx = _result(dx, (rows, K), dy.dtype, dy, "dx")
    _contiguous(dy, w, dx)
    _call("swiglu_grouped_mm_dgrad", dy, stream, dy.data_ptr(), w.data_ptr(), ends.data_ptr(), dx.data_ptr(), rows, E,
          N, K, SWIGLU_BF16)
    return dx


def swiglu_grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, ends: torch.Tensor, dw: torch.Tensor = None,
                            accumulate: bool = False, dtype: torch.dtype = None, stream=None) -> torch.Tensor:
    """dW[e] = sum over the group's rows of dy[t]^T x[t]: dy [rows, N], x [rows, K]
    -> dw [E, N, K] of ``dtype`` (bfloat16, the default, or float32; that of ``dw``
    when one is given).  ``accumulate`` adds to a float32 ``dw``."""
    _check_cuda(dy, x)
    if dy.dtype != torch.bfloat16:
        raise ValueError("the grouped products take bfloat16 tensors")
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [rows, N] and x [rows, K] over the same rows")
    if dtype is None:
        dtype = dw.dtype if dw is not None else torch.bfloat16
    if dtype not in _DTYPE:
        raise ValueError("dw must be float32 or bfloat16")
    if accumulate and (dw is None or dtype != torch.float32):
        raise ValueError("accumulate adds to a float32 dw: give one")
    (rows, N), K, E = dy.shape, x.shape[1], ends.numel()
    _ends(ends, dy, E)
    dw = _result(dw, (E, N, K), dtype, dy, "dw")
    _contiguous(dy, x, dw)
    _call("swiglu_grouped_mm_wgrad", dy, stream, dy.data_ptr(), x.data_ptr(), ends.data_ptr(), dw.data_ptr(), rows, E,
          N, K, SWIGLU_BF16, _DTYPE[dtype], 1 if accumulate else 0)
    return dw


def grouped_timeout_flag() -> int:
    """1 if any grouped product so far gave up on an internal wait, else 0
    (synchronises with the current device)."""
    out = ctypes.c_int(0)
    st = lib.swiglu_grouped_timeout_flag(ctypes.byref(out))
    if st != 0:
        raise SwigluError(st, "swiglu_grouped_timeout_flag")
    return int(out.value)


__all__ = ["swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_grouped_fc1_fwd", "swiglu_grouped_mm_fwd",
           "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "grouped_timeout_flag", "CKPT8_BLOCK", "MAX_GROUPS",
           "MOE_EXPORTS"]
