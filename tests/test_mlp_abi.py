"""Host-side tests of the layer norm and the 4-bit MLP: headers and library agree, bad
arguments are refused before the GPU is touched (these run on a machine without one;
pointers are plain integers that are never dereferenced), and the Python layer's checks."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = {"MX4_EXPORTS": "swiglu_mx4.h", "NORM_EXPORTS": "swiglu_norm.h"}
OK, NULL, DTYPE, SHAPE, STRIDE, ALIAS, WORKSPACE = 0, -1, -2, -3, -4, -5, -7
F32, BF16 = 0, 1
# fake device addresses, 256-byte aligned and far apart
A, B, C, D, E, F, G, H, I = (0x10_0000_0000 * i for i in range(1, 10))
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def sw():
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


@pytest.mark.parametrize("exports,name", HEADERS.items())
def test_header_and_library_agree(sw, exports, name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)
    declared = set(re.findall(r"\b(swiglu_[a-z0-9_]+)\s*\(", text))
    assert declared == set(getattr(sw, exports))
    for f in declared:
        assert hasattr(sw.lib, f)


def define(name, header):
    return int(re.search(rf"#define {name} (\d+)\n", open(os.path.join(ROOT, "include", header)).read()).group(1))


def test_block(sw):
    assert define("SWIGLU_MX4_BLOCK", "swiglu_mx4.h") == sw.MX4_BLOCK


@pytest.mark.parametrize("name", ["swiglu_mx4.h", "swiglu_norm.h"])
def test_headers_compile_as_c(tmp_path, name):
    src = tmp_path / "h.c"
    src.write_text(f'#include "{name}"\nint main(void) {{ return 0; }}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


# ------------------------------------------------------------------ layer norm ---

def fwd(sw, x=A, w=B, b=C, y=D, mean=E, rstd=F, rows=4, n=64, sx=64, sy=64, eps=1e-5, dt=BF16, pt=BF16):
    return sw.lib.swiglu_layer_norm_fwd(x, w, b, y, mean, rstd, rows, n, sx, sy, eps, dt, pt, None)


def bwd(sw, dy=A, x=B, mean=C, rstd=D, w=E, dx=F, dw=G, db=H, ws=I, wsb=1 << 30, rows=4, n=64, sdy=64, sx=64, sdx=64,
        dt=BF16, pt=BF16):
    return sw.lib.swiglu_layer_norm_bwd(dy, x, mean, rstd, w, dx, dw, db, ws, wsb, rows, n, sdy, sx, sdx, dt, pt, None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (DTYPE, dict(pt=2)), (DTYPE, dict(dt=F32)), (DTYPE, dict(dt=-1)), (SHAPE, dict(rows=-1)),
    (SHAPE, dict(n=-1)), (SHAPE, dict(rows=1 << 31)), (SHAPE, dict(n=(1 << 30) + 1)), (SHAPE, dict(eps=-1e-9)),
    (SHAPE, dict(eps=INF)), (SHAPE, dict(eps=NAN)), (OK, dict(rows=0, x=0, y=0)), (OK, dict(n=0, x=0, y=0)),
    (NULL, dict(x=0)), (NULL, dict(y=0)), (STRIDE, dict(sx=63)), (STRIDE, dict(sy=63)), (STRIDE, dict(x=A + 1)),
    (STRIDE, dict(y=D + 1)), (STRIDE, dict(w=B + 1)), (STRIDE, dict(b=C + 2, pt=F32)), (STRIDE, dict(mean=E + 2)),
    (STRIDE, dict(rstd=F + 1)), (ALIAS, dict(y=A)), (ALIAS, dict(y=A + 100)), (ALIAS, dict(y=B)), (ALIAS, dict(y=C)),
    (ALIAS, dict(mean=A)), (ALIAS, dict(rstd=E + 4)), (ALIAS, dict(mean=D + 8)), (SHAPE, dict(rows=1 << 30, sx=1 << 40))])
def test_layer_norm_fwd_refusals(sw, status, kw):
    assert fwd(sw, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (DTYPE, dict(pt=7)), (DTYPE, dict(dt=F32)), (SHAPE, dict(rows=-1)), (SHAPE, dict(n=-1)),
    (SHAPE, dict(rows=1 << 31)), (OK, dict(n=0, dy=0, x=0, dx=0)), (OK, dict(rows=0, dy=0, dw=0, db=0)),
    (STRIDE, dict(rows=0, dw=G + 1)), (NULL, dict(dy=0)), (NULL, dict(x=0)), (NULL, dict(mean=0)), (NULL, dict(rstd=0)),
    (NULL, dict(dx=0)), (STRIDE, dict(sdy=63)), (STRIDE, dict(sx=63)), (STRIDE, dict(sdx=63)), (STRIDE, dict(dy=A + 1)),
    (STRIDE, dict(dx=F + 1)), (STRIDE, dict(db=H + 1)), (STRIDE, dict(mean=C + 1)), (ALIAS, dict(dx=A)),
    (ALIAS, dict(dx=B + 64)), (ALIAS, dict(dw=E)), (ALIAS, dict(dw=H)), (ALIAS, dict(db=F)), (ALIAS, dict(dx=C))])
def test_layer_norm_bwd_refusals(sw, status, kw):
    assert bwd(sw, **kw) == status


def test_layer_norm_sizes_and_flags_refuse(sw):
    size = ctypes.c_size_t(7)
    f = sw.lib.swiglu_layer_norm_bwd_workspace_size
    assert f(4, 4, BF16, None) == NULL and f(4, 4, 5, ctypes.byref(size)) == DTYPE
    assert f(-1, 4, BF16, ctypes.byref(size)) == SHAPE and f(4, 1 << 31, BF16, ctypes.byref(size)) == SHAPE
    assert f(0, 4, BF16, ctypes.byref(size)) == OK and size.value == 0
    assert sw.lib.swiglu_layer_norm_timeout_flag(None) == NULL
    assert define("SWIGLU_NORM_MAX_ROWS", "swiglu_norm.h") == (1 << 31) - 1


# -------------------------------------------------------------------- 4 bits ---

def quantize(sw, x=A, q=B, s=C, rows=4, n=64, parts=1, sx=64, dt=BF16):
    return sw.lib.swiglu_mx4_quantize(x, q, s, rows, n, parts, sx, dt, None)


def dequantize(sw, q=A, s=B, y=C, rows=4, n=64, parts=1, sy=64, dt=BF16):
    return sw.lib.swiglu_mx4_dequantize(q, s, y, rows, n, parts, sy, dt, None)


def mm(sw, xq=A, xs=B, wq=C, ws=D, y=E, M=4, N=16, K=64, dt=BF16):
    return sw.lib.swiglu_mx4_mm_fwd(xq, xs, wq, ws, y, M, N, K, dt, None)


def mlp(sw, x=A, w1q=B, w1s=C, w2q=D, w2s=E, out=F, ws=G, wsb=1 << 30, M=4, h=64, n=32, N=64, sx=64, dt=BF16):
    return sw.lib.swiglu_mx4_mlp_fwd(x, w1q, w1s, w2q, w2s, out, ws, wsb, M, h, n, N, sx, dt, None)


BIG = 2147483136


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(rows=-1)), (SHAPE, dict(n=-1)), (SHAPE, dict(rows=BIG + 1)),
    (SHAPE, dict(n=(1 << 30) + 1)), (SHAPE, dict(parts=0)), (SHAPE, dict(parts=3)), (OK, dict(rows=0, x=0, q=0, s=0)),
    (OK, dict(n=0, x=0, q=0, s=0)), (NULL, dict(x=0)), (NULL, dict(q=0)), (NULL, dict(s=0)), (STRIDE, dict(sx=63)),
    (STRIDE, dict(x=A + 1)), (STRIDE, dict(x=A + 2, dt=F32)), (STRIDE, dict(q=B + 8)), (STRIDE, dict(s=C + 8)),
    (ALIAS, dict(q=A)), (ALIAS, dict(s=A + 64)), (ALIAS, dict(s=B + 64)), (ALIAS, dict(s=B - 256))])
def test_quantize_refusals(sw, status, kw):
    assert quantize(sw, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=-1)), (SHAPE, dict(rows=-1)), (SHAPE, dict(n=-1)), (SHAPE, dict(parts=-1)), (SHAPE, dict(parts=3)),
    (OK, dict(rows=0, y=0)), (OK, dict(n=0, y=0)), (NULL, dict(q=0)), (NULL, dict(s=0)), (NULL, dict(y=0)),
    (STRIDE, dict(sy=63)), (STRIDE, dict(y=C + 1)), (STRIDE, dict(q=A + 4)), (STRIDE, dict(s=B + 2)), (ALIAS, dict(y=A)),
    (ALIAS, dict(y=B + 2))])
def test_dequantize_refusals(sw, status, kw):
    assert dequantize(sw, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=F32)), (SHAPE, dict(M=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(K=-1)), (SHAPE, dict(M=BIG + 1)),
    (SHAPE, dict(N=BIG + 1)), (SHAPE, dict(K=(1 << 30) + 1)), (OK, dict(M=0, xq=0, y=0)), (OK, dict(N=0, wq=0, y=0)),
    (NULL, dict(y=0)), (NULL, dict(K=0, y=0)), (NULL, dict(xq=0)), (NULL, dict(xs=0)), (NULL, dict(wq=0)),
    (NULL, dict(ws=0)), (STRIDE, dict(y=E + 1)), (STRIDE, dict(xq=A + 8)), (STRIDE, dict(ws=D + 8)), (ALIAS, dict(y=A)),
    (ALIAS, dict(y=B + 16)), (ALIAS, dict(y=C)), (ALIAS, dict(y=D)), (SHAPE, dict(M=BIG, N=1 << 20))])
def test_mx4_mm_refusals(sw, status, kw):
    assert mm(sw, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(M=-1)), (SHAPE, dict(h=-1)), (SHAPE, dict(n=-1)), (SHAPE, dict(N=-1)),
    (SHAPE, dict(M=BIG + 1)), (SHAPE, dict(n=BIG // 2 + 1)), (OK, dict(M=0, x=0, out=0)), (OK, dict(N=0, out=0)),
    (NULL, dict(out=0)), (NULL, dict(x=0)), (NULL, dict(w1q=0)), (NULL, dict(w1s=0)), (NULL, dict(w2q=0)),
    (NULL, dict(w2s=0)), (STRIDE, dict(sx=63)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws=G + 8)),
    (WORKSPACE, dict(wsb=100)), (ALIAS, dict(out=A)), (ALIAS, dict(out=D)), (ALIAS, dict(ws=B)), (ALIAS, dict(ws=F)),
    (ALIAS, dict(out=G + 64)), (STRIDE, dict(x=A + 1)), (STRIDE, dict(w1q=B + 8)), (STRIDE, dict(w2s=E + 4)),
    (STRIDE, dict(out=F + 1))])
def test_mx4_mlp_refusals(sw, status, kw):
    assert mlp(sw, **kw) == status


def test_mx4_sizes(sw):
    size = ctypes.c_size_t(0)
    f, g = sw.lib.swiglu_mx4_scales_size, sw.lib.swiglu_mx4_mlp_workspace_size
    assert f(1, 1, 1, None) == NULL and f(3, 1, 2, ctypes.byref(size)) == SHAPE and f(1, -1, 1, ctypes.byref(size)) == SHAPE
    for rows, n, parts, want in ((1, 1, 1, 512), (128, 128, 1, 512), (129, 129, 1, 2048), (258, 128, 2, 2048), (0, 64, 1, 0)):
        assert f(rows, n, parts, ctypes.byref(size)) == OK and size.value == want
        shape = sw.mx4_scales_shape(rows, n, parts)
        assert shape[0] * shape[1] * shape[2] == want
    assert g(1, 1, 1, None) == NULL and g(-1, 1, 1, ctypes.byref(size)) == SHAPE
    assert g(1, 64, 64, ctypes.byref(size)) == OK and size.value == 2 * (256 + 512)
    assert sw.mx4_mlp_workspace_bytes(1, 64, 64) == size.value
    assert sw.lib.swiglu_mx4_timeout_flag(None) == NULL
    with pytest.raises(ValueError, match="multiple of parts"):
        sw.mx4_scales_shape(3, 64, 2)
    assert define("SWIGLU_MX4_MAX_ROWS", "swiglu_mx4.h") == BIG
    assert define("SWIGLU_MX4_MAX_COLS", "swiglu_mx4.h") == 1 << 30


# -------------------------------------------------------------- Python layer ---

def test_python_layer_refuses_cpu_tensors_and_wrong_arguments(sw):
    x = torch.zeros(4, 64).bfloat16()
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    for call in (lambda: sw.swiglu_layer_norm_fwd(x), lambda: sw.swiglu_layer_norm_bwd(x, x, x[:, 0], x[:, 0]),
                 lambda: sw.swiglu_mx4_quantize(x), lambda: sw.swiglu_mx4_dequantize(q, s, 64),
                 lambda: sw.swiglu_mx4_mm_fwd(q, s, q, s), lambda: sw.swiglu_mx4_mlp_fwd(x, q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="uint8"):
        sw.swiglu_mx4_mm_fwd(q.int(), s, q, s)
    with pytest.raises(ValueError, match="float8_e8m0fnu"):
        sw.swiglu_mx4_dequantize(q, s.view(torch.uint8), 64)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sw.layer_norm_bwd_workspace_bytes(4, 64, torch.float16)


def test_modules_refuse_wrong_shapes(sw):
    from gate_up_swiglu_gb300.mlp import LayerNorm, Mx4SwiGLU

    with pytest.raises(ValueError, match="64"):
        LayerNorm(64)(torch.zeros(2, 32))
    m = Mx4SwiGLU(64, 40)
    assert m.w1_q.shape == (80, 32) and m.w2_q.shape == (64, 32) and m.w1_scales.shape == (2, 1, 512)
    with pytest.raises(ValueError, match="64"):
        m(torch.zeros(2, 32))
    with pytest.raises(NotImplementedError, match="no backward"):
        m(torch.zeros(2, 64, requires_grad=True))
    with pytest.raises(ValueError, match="2n"):
        Mx4SwiGLU.from_weights(torch.zeros(10, 8), torch.zeros(8, 4))


def test_mx4_module_refuses_tangents(sw):
    import torch.autograd.forward_ad as fw
    from gate_up_swiglu_gb300.mlp import Mx4SwiGLU

    m, x = Mx4SwiGLU(64, 40), torch.zeros(2, 64)
    with fw.dual_level(), torch.no_grad():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            m(fw.make_dual(x, x))


def test_a_torch_without_the_scale_type_keeps_the_rest(sw):
    code = """
import torch
del torch.float8_e8m0fnu
import gate_up_swiglu_gb300 as sw
from gate_up_swiglu_gb300.mlp import LayerNorm, Mx4SwiGLU
x = torch.zeros(4, 16).bfloat16()
LayerNorm(16)
try:
    sw.swiglu_layer_norm_fwd(x)
    assert False
except ValueError as e:
    assert "CUDA" in str(e)
for fn in (lambda: sw.swiglu_mx4_quantize(x), lambda: sw.swiglu_mx4_dequantize(x, x, 16), lambda: sw.swiglu_mx4_mm_fwd(x, x, x, x),
           lambda: sw.swiglu_mx4_mlp_fwd(x, x, x, x, x), lambda: sw.mx4_scale_rows(x, 4, 16), lambda: Mx4SwiGLU(16, 16)):
    try:
        fn()
        assert False
    except NotImplementedError as e:
        assert "float8" in str(e)
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
