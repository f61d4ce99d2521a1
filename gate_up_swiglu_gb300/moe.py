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

from . import (_DTYPE, SWIGLU_BF16, SwigluError, _on_device, _raw_stream, _rows_view, _stream_handle, lib)

CKPT8_BLOCK = 32
MAX_GROUPS = 1024
# None where torch has no such type: the other operators work all the same
Q_DTYPE = getattr(torch, "float8_e4m3fn", None)
SCALE_DTYPE = getattr(torch, "float8_e8m0fnu", None)

# every symbol include/swiglu_moe.h declares
MOE_EXPORTS = ("swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_grouped_fc1_fwd", "swiglu_grouped_mm_fwd",
               "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "swiglu_grouped_slices",
               "swiglu_grouped_timeout_flag")


def _declare() -> None:
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name, args in (
            ("swiglu_ckpt8_fwd", [vp] * 5 + [i64] * 6 + [i32, vp]),
            ("swiglu_ckpt8_bwd", [vp] * 7 + [i64] * 7 + [i32, vp]),
            ("swiglu_grouped_fc1_fwd", [vp] * 8 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_fwd", [vp] * 4 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_dgrad", [vp] * 4 + [i64] * 4 + [i32, vp]),
            ("swiglu_grouped_mm_wgrad", [vp] * 4 + [i64] * 4 + [i32, i32, i32, vp]),
            ("swiglu_grouped_slices", [i32] + [i64] * 4 + [i32, ctypes.POINTER(ctypes.c_int)]),
            ("swiglu_grouped_timeout_flag", [ctypes.POINTER(ctypes.c_int)])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i32


_declare()


# the current device without the check that CUDA is initialised (these calls
# have CUDA tensors in hand)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name: str, fn, t: torch.Tensor, stream, *args) -> None:
    index = t.get_device()
    if stream is None and index == _current_device():  # the common case, without a context switch
        st = fn(*args, _raw_stream(index) if _raw_stream is not None else _stream_handle(t, None))
    else:
        with _on_device(t.device):
            st = fn(*args, _stream_handle(t, stream))
    if st != 0:
        raise SwigluError(st, name)


def _rows(t: torch.Tensor, cols: int, name: str):
    """(rows, row stride) of a [..., cols] tensor (cols its last dimension)."""
    if cols and t.is_contiguous():
        return t.numel() // cols, cols
    rows, _, stride = _rows_view(t, name)
    return rows, stride


def _given(t: torch.Tensor, rows: int, cols: int, dtype, device, name: str) -> int:
    """The row stride of a tensor the caller gave, checked to be [rows, cols]."""
    if t.device != device:
        raise ValueError("all tensors must be on the same CUDA device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    r, c, stride = _rows_view(t, name)
    if (r, c) != (rows, cols):
        raise ValueError(f"{name} must have {rows} rows of {cols}")
    return stride


def _weights(w: torch.Tensor, rows: int, device, name: str) -> int:
    """The address of an fp32 vector with one value per row."""
    if w.dtype is not _F32 or w.numel() != rows or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {torch.float32} tensor of {rows} elements")
    if w.device != device:
        raise ValueError("all tensors must be on the same CUDA device")
    return w.data_ptr()


def _float_type(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("libswiglu operates on CUDA tensors only")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError("tensors must all be float32 or all bfloat16")
    return code


def _need_checkpoint_types() -> None:
    if Q_DTYPE is None or SCALE_DTYPE is None:
        raise NotImplementedError("the 8-bit checkpoint needs a torch with float8_e4m3fn and float8_e8m0fnu")


def swiglu_ckpt8_fwd(x: torch.Tensor, w: torch.Tensor = None, y: torch.Tensor = None, q: torch.Tensor = None,
                     scales: torch.Tensor = None, stream=None):
    """(y, q, scales): y = w[row] * silu(gate) * up and the 8-bit checkpoint of x.

    ``w`` (fp32, one weight per row of x) is optional."""
    _need_checkpoint_types()
    shape, dtype, device = x.shape, x.dtype, x.device
    two_n = shape[-1]
    if two_n % 2:
        raise ValueError("x's last dimension must be even (gate and up halves)")
    n, lead = two_n // 2, shape[:-1]
    cols = 2 * ((n + CKPT8_BLOCK - 1) // CKPT8_BLOCK)
    code = _float_type(x)
    rows, sx = _rows(x, two_n, "x")
    sy, sq, ss = n, two_n, cols
    if y is None:
        y = torch.empty((*lead, n), dtype=dtype, device=device)
    else:
        sy = _given(y, rows, n, dtype, device, "y")
    if q is None:
        q = torch.empty(shape, dtype=Q_DTYPE, device=device)
    else:
        sq = _given(q, rows, two_n, Q_DTYPE, device, "q")
    if scales is None:
        scales = torch.empty((*lead, cols), dtype=SCALE_DTYPE, device=device)
    else:
        ss = _given(scales, rows, cols, SCALE_DTYPE, device, "scales")
    _call("swiglu_ckpt8_fwd", lib.swiglu_ckpt8_fwd, x, stream, x.data_ptr(),
          None if w is None else _weights(w, rows, device, "w"), y.data_ptr(), q.data_ptr(), scales.data_ptr(), rows, n,
          sx, sy, sq, ss, code)
    return y, q, scales


def swiglu_ckpt8_bwd(dy: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, w: torch.Tensor = None,
                     dx: torch.Tensor = None, dw: torch.Tensor = None, y: torch.Tensor = None,
                     return_y: bool = False, stream=None):
    """(dx, dw, y) of the SwiGLU at the checkpointed x: the input gradient, the
    fp32 gradient of the row weights (None without ``w``) and, with ``return_y``
    (or a ``y`` given), the forward's output made again from the checkpoint
    (else None)."""
    _need_checkpoint_types()
    if w is None and dw is not None:
        raise ValueError("dw is the gradient of w: it needs w")
    shape, dtype, device = dy.shape, dy.dtype, dy.device
    n = shape[-1]
    two_n, cols = 2 * n, 2 * ((n + CKPT8_BLOCK - 1) // CKPT8_BLOCK)
    code = _float_type(dy)
    rows, sdy = _rows(dy, n, "dy")
    if q.dtype != Q_DTYPE or scales.dtype != SCALE_DTYPE:
        raise ValueError("a checkpoint is q (float8_e4m3fn) and scales (float8_e8m0fnu)")
    if q.device != device or scales.device != device:
        raise ValueError("all tensors must be on the same CUDA device")
    (qrows, sq), (srows, ss) = _rows(q, q.shape[-1], "q"), _rows(scales, scales.shape[-1], "scales")
    if qrows != rows or srows != rows or q.shape[-1] != two_n or scales.shape[-1] != cols:
        raise ValueError(f"the checkpoint of [{rows}, {two_n}] is q [{rows}, {two_n}] and scales [{rows}, {cols}]")
    sdx, sy = two_n, n
    if dx is None:
        dx = torch.empty((*shape[:-1], two_n), dtype=dtype, device=device)
    else:
        sdx = _given(dx, rows, two_n, dtype, device, "dx")
    if y is not None:
        sy = _given(y, rows, n, dtype, device, "y")
    elif return_y:
        y = torch.empty(shape, dtype=dtype, device=device)
    wp = dwp = None
    if w is not None:
        wp = _weights(w, rows, device, "w")
        if dw is None:
            dw = torch.empty(w.shape, dtype=torch.float32, device=device)
            dwp = dw.data_ptr()
        else:
            dwp = _weights(dw, rows, device, "dw")
    _call("swiglu_ckpt8_bwd", lib.swiglu_ckpt8_bwd, dy, stream, dy.data_ptr(), q.data_ptr(), scales.data_ptr(), wp,
          dx.data_ptr(), dwp, _ptr(y), rows, n, sdy, sq, ss, sdx, sy, code)
    return dx, dw, y


def _check_products(a: torch.Tensor, b: torch.Tensor, ends: torch.Tensor) -> None:
    """Checks shared by the products: two contiguous bf16 tensors on one CUDA device."""
    device = a.get_device()
    if device < 0 or b.get_device() < 0:
        raise ValueError("libswiglu operates on CUDA tensors only")
    if a.dtype is not _BF16 or b.dtype is not _BF16:
        raise ValueError("the grouped products take bfloat16 tensors")
    if b.get_device() != device or ends.get_device() != device:
        raise ValueError("all tensors must be on the same CUDA device")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("the grouped products need contiguous tensors")


def _rows_and_experts(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, name: str):
    """The shapes of rows x [rows, *] and w [E, N, K]."""
    _check_products(x, w, ends)
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != 3:
        raise ValueError(f"{name} must have two dimensions and w three: [experts, N, K]")
    _check_ends(ends, ws[0])
    return xs, ws


def _check_ends(ends: torch.Tensor, groups: int) -> None:
    if ends.dtype is not _I32 or ends.numel() != groups or not ends.is_contiguous():
        raise ValueError(f"ends must be a contiguous {torch.int32} tensor of {groups} elements")


def _result(t, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {like.device}")
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
    if (fc1 is not None and save != "bf16") or ((q is not None or scales is not None) and save != "fp8"):
        raise ValueError('fc1 is written with save="bf16", q and scales with save="fp8"')
    if save == "fp8":
        _need_checkpoint_types()
    (rows, K), (E, two_n, wk) = _rows_and_experts(x, w, ends, "x")
    if wk != K or two_n % 2:
        raise ValueError("w must be [experts, 2n, K] with x's K")
    n = two_n // 2
    nb = -(-n // CKPT8_BLOCK)
    y = _result(y, (rows, n), x.dtype, x, "y")
    fc1 = _result(fc1, (rows, two_n), x.dtype, x, "fc1") if save == "bf16" else None
    q = _result(q, (rows, two_n), Q_DTYPE, x, "q") if save == "fp8" else None
    scales = _result(scales, (rows, 2 * nb), SCALE_DTYPE, x, "scales") if save == "fp8" else None
    _call("swiglu_grouped_fc1_fwd", lib.swiglu_grouped_fc1_fwd, x, stream, x.data_ptr(), w.data_ptr(), ends.data_ptr(),
          None if probs is None else _weights(probs, rows, x.device, "probs"), y.data_ptr(), _ptr(fc1), _ptr(q),
          _ptr(scales), rows, E, n, K, SWIGLU_BF16)
    return (y, fc1) if save == "bf16" else (y, q, scales) if save == "fp8" else y


def swiglu_grouped_mm_fwd(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, y: torch.Tensor = None,
                          stream=None) -> torch.Tensor:
    """y[t] = W[e] x[t]: x [rows, K], w [E, N, K] -> y [rows, N]."""
    (rows, K), (E, N, wk) = _rows_and_experts(x, w, ends, "x")
    if wk != K:
        raise ValueError("w must be [experts, N, K] with x's K")
    y = _result(y, (rows, N), x.dtype, x, "y")
    _call("swiglu_grouped_mm_fwd", lib.swiglu_grouped_mm_fwd, x, stream, x.data_ptr(), w.data_ptr(), ends.data_ptr(),
          y.data_ptr(), rows, E, N, K, SWIGLU_BF16)
    return y


def swiglu_grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, dx: torch.Tensor = None,
                            stream=None) -> torch.Tensor:
    """dx[t] = W[e]^T dy[t]: dy [rows, N], w [E, N, K] -> dx [rows, K]."""
    (rows, N), (E, wn, K) = _rows_and_experts(dy, w, ends, "dy")
    if wn != N:
        raise ValueError("w must be [experts, N, K] with dy's N")
    dx = _result(dx, (rows, K), dy.dtype, dy, "dx")
    _call("swiglu_grouped_mm_dgrad", lib.swiglu_grouped_mm_dgrad, dy, stream, dy.data_ptr(), w.data_ptr(),
          ends.data_ptr(), dx.data_ptr(), rows, E, N, K, SWIGLU_BF16)
    return dx


def swiglu_grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, ends: torch.Tensor, dw: torch.Tensor = None,
                            accumulate: bool = False, dtype: torch.dtype = None, stream=None) -> torch.Tensor:
    """dW[e] = sum over the group's rows of dy[t]^T x[t]: dy [rows, N], x [rows, K]
    -> dw [E, N, K] of ``dtype`` (bfloat16, the default, or float32; that of ``dw``
    when one is given).  ``accumulate`` adds to a float32 ``dw``."""
    _check_products(dy, x, ends)
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [rows, N] and x [rows, K] over the same rows")
    if dtype is None:
        dtype = dw.dtype if dw is not None else torch.bfloat16
    if dtype not in _DTYPE:
        raise ValueError("dw must be float32 or bfloat16")
    if accumulate and (dw is None or dtype != torch.float32):
        raise ValueError("accumulate adds to a float32 dw: give one")
    (rows, N), K, E = dy.shape, x.shape[1], ends.numel()
    _check_ends(ends, E)
    dw = _result(dw, (E, N, K), dtype, dy, "dw")
    _call("swiglu_grouped_mm_wgrad", lib.swiglu_grouped_mm_wgrad, dy, stream, dy.data_ptr(), x.data_ptr(),
          ends.data_ptr(), dw.data_ptr(), rows, E, N, K, SWIGLU_BF16, _DTYPE[dtype], 1 if accumulate else 0)
    return dw


_PRODUCTS = ("fc1", "mm", "dgrad", "wgrad")


def grouped_slices(product: str, rows: int, groups: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """How a product ("fc1", with n as N, "mm", "dgrad" or "wgrad") of these sizes is
    computed: 0, pairs of CTAs; else the CTAs that share a tile's contraction.
    ``dtype`` is that of a weight gradient."""
    if product not in _PRODUCTS:
        raise ValueError(f"product must be one of {_PRODUCTS}")
    if dtype not in _DTYPE:
        raise ValueError("dtype must be float32 or bfloat16")
    out = ctypes.c_int(0)
    st = lib.swiglu_grouped_slices(_PRODUCTS.index(product), rows, groups, N, K, _DTYPE[dtype], ctypes.byref(out))
    if st != 0:
        raise SwigluError(st, "swiglu_grouped_slices")
    return int(out.value)


def grouped_timeout_flag() -> int:
    """1 if any grouped product so far gave up on an internal wait, else 0
    (synchronises with the current device)."""
    out = ctypes.c_int(0)
    st = lib.swiglu_grouped_timeout_flag(ctypes.byref(out))
    if st != 0:
        raise SwigluError(st, "swiglu_grouped_timeout_flag")
    return int(out.value)


__all__ = ["swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_grouped_fc1_fwd", "swiglu_grouped_mm_fwd",
           "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "grouped_slices", "grouped_timeout_flag", "CKPT8_BLOCK",
           "MAX_GROUPS", "MOE_EXPORTS"]
