"""Host-side tests of the routed experts' operators: the header and the library
agree, bad arguments are refused before the GPU is touched (these run on a
machine without one; pointers are plain integers that are never dereferenced),
and the Python layer's checks."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "swiglu_moe.h")
OK, NULL, DTYPE, SHAPE, STRIDE, ALIAS = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
# fake device addresses, 256-byte aligned and far apart
A, B, C, D, E, F, G = (0x10_0000_0000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def sw():
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


def test_header_and_library_agree(sw):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(swiglu_[a-z0-9_]+)\s*\(", text))
    assert declared == set(sw.MOE_EXPORTS)
    for name in declared:
        assert hasattr(sw.lib, name)
    assert f"SWIGLU_MAX_GROUPS {sw.MAX_GROUPS}\n" in open(HEADER).read()
    assert f"SWIGLU_CKPT8_BLOCK {sw.CKPT8_BLOCK}\n" in open(HEADER).read()


def ckpt8_fwd(sw, x=A, w=0, y=B, q=C, s=D, rows=4, n=64, sx=128, sy=64, sq=128, ss=4, dt=BF16):
    return sw.lib.swiglu_ckpt8_fwd(x, w, y, q, s, rows, n, sx, sy, sq, ss, dt, None)


def ckpt8_bwd(sw, dy=A, q=B, s=C, w=D, dx=E, dw=F, y=G, rows=4, n=64, sdy=64, sq=128, ss=4, sdx=128, sy=64, dt=BF16):
    return sw.lib.swiglu_ckpt8_bwd(dy, q, s, w, dx, dw, y, rows, n, sdy, sq, ss, sdx, sy, dt, None)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (DTYPE, dict(dt=-1)), (SHAPE, dict(rows=-1)), (SHAPE, dict(n=-1)),
    (SHAPE, dict(n=(1 << 30) + 1)), (SHAPE, dict(rows=1 << 40)), (OK, dict(rows=0, x=0, y=0, q=0, s=0)),
    (OK, dict(n=0, x=0, y=0, q=0, s=0)), (NULL, dict(x=0)), (NULL, dict(y=0)), (NULL, dict(q=0)), (NULL, dict(s=0)),
    (STRIDE, dict(sx=127)), (STRIDE, dict(sy=63)), (STRIDE, dict(sq=127)), (STRIDE, dict(ss=3)),
    (ALIAS, dict(y=A)), (ALIAS, dict(q=A + 100)), (ALIAS, dict(s=B)), (ALIAS, dict(w=B)), (ALIAS, dict(s=C + 8)),
    (STRIDE, dict(x=A + 1)), (STRIDE, dict(y=B + 1)), (STRIDE, dict(w=G + 2)), (STRIDE, dict(x=A + 2, dt=F32))])
def test_ckpt8_fwd_refusals(sw, status, kw):
    assert ckpt8_fwd(sw, **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=7)), (SHAPE, dict(rows=-3)), (SHAPE, dict(n=-1)), (OK, dict(rows=0, dy=0, q=0, s=0, dx=0)),
    (OK, dict(n=0, dw=0, dy=0)), (STRIDE, dict(n=0, dw=F + 1)), (NULL, dict(dy=0)), (NULL, dict(q=0)),
    (NULL, dict(s=0)), (NULL, dict(dx=0)), (NULL, dict(w=0)), (NULL, dict(dw=0)), (STRIDE, dict(sdy=63)),
    (STRIDE, dict(sq=1)), (STRIDE, dict(ss=3)), (STRIDE, dict(sdx=127)), (STRIDE, dict(sy=63)),
    (ALIAS, dict(dx=A)), (ALIAS, dict(y=E)), (ALIAS, dict(dw=D)), (ALIAS, dict(y=B)), (ALIAS, dict(dw=E)),
    (STRIDE, dict(dy=A + 1)), (STRIDE, dict(dx=E + 1)), (STRIDE, dict(y=G + 1)), (STRIDE, dict(dw=F + 2))])
def test_ckpt8_bwd_refusals(sw, status, kw):
    assert ckpt8_bwd(sw, **kw) == status


def fc1(sw, x=A, w=B, ends=C, probs=0, y=D, fc1=0, q=0, s=0, rows=10, groups=3, n=16, K=32, dt=BF16):
    return sw.lib.swiglu_grouped_fc1_fwd(x, w, ends, probs, y, fc1, q, s, rows, groups, n, K, dt, None)


def mm(sw, which, x=A, w=B, ends=C, y=D, rows=10, groups=3, N=16, K=32, dt=BF16):
    return getattr(sw.lib, "swiglu_grouped_mm_" + which)(x, w, ends, y, rows, groups, N, K, dt, None)


def wgrad(sw, dy=A, x=B, ends=C, dw=D, rows=10, groups=3, N=16, K=32, dt=BF16, dwt=BF16, acc=0):
    return sw.lib.swiglu_grouped_mm_wgrad(dy, x, ends, dw, rows, groups, N, K, dt, dwt, acc, None)


SIZES = [(DTYPE, dict(dt=F32)), (DTYPE, dict(dt=5)), (SHAPE, dict(rows=-1)), (SHAPE, dict(rows=1 << 31)),
         (SHAPE, dict(groups=0)), (SHAPE, dict(groups=1025)), (SHAPE, dict(K=0)), (SHAPE, dict(K=12)),
         (SHAPE, dict(K=-8)), (SHAPE, dict(K=1 << 31))]


@pytest.mark.parametrize("status,kw", SIZES + [
    (SHAPE, dict(n=0)), (SHAPE, dict(n=12)), (SHAPE, dict(n=1 << 30)), (OK, dict(rows=0, x=0, y=0, ends=0)),
    (NULL, dict(x=0)), (NULL, dict(w=0)), (NULL, dict(ends=0)), (NULL, dict(y=0)), (NULL, dict(q=E)),
    (NULL, dict(s=E)), (ALIAS, dict(fc1=E, q=F, s=G)), (ALIAS, dict(y=A)), (ALIAS, dict(fc1=D)),
    (ALIAS, dict(q=D, s=F)), (ALIAS, dict(q=E, s=E + 32)), (ALIAS, dict(probs=D)), (STRIDE, dict(x=A + 8)),
    (STRIDE, dict(y=D + 2)), (STRIDE, dict(ends=C + 2)), (STRIDE, dict(probs=G + 1)), (STRIDE, dict(fc1=E + 8)),
    (STRIDE, dict(q=E + 8, s=F))])
def test_fc1_refusals(sw, status, kw):
    assert fc1(sw, **kw) == status


@pytest.mark.parametrize("which", ["fwd", "dgrad"])
@pytest.mark.parametrize("status,kw", SIZES + [
    (SHAPE, dict(N=0)), (SHAPE, dict(N=20)), (SHAPE, dict(N=1 << 30)), (OK, dict(rows=0, x=0, y=0, ends=0)),
    (NULL, dict(x=0)), (NULL, dict(w=0)), (NULL, dict(ends=0)), (NULL, dict(y=0)), (ALIAS, dict(y=A)),
    (ALIAS, dict(y=B + 64)), (ALIAS, dict(y=C)), (STRIDE, dict(x=A + 8)), (STRIDE, dict(w=B + 4)),
    (STRIDE, dict(y=D + 2)), (STRIDE, dict(ends=C + 1))])
def test_mm_refusals(sw, which, status, kw):
    assert mm(sw, which, **kw) == status


@pytest.mark.parametrize("status,kw", SIZES + [
    (SHAPE, dict(N=0)), (DTYPE, dict(dwt=2)), (DTYPE, dict(acc=1)), (NULL, dict(dy=0)), (NULL, dict(x=0)),
    (NULL, dict(ends=0)), (NULL, dict(dw=0)), (NULL, dict(rows=0, dw=0)), (OK, dict(rows=0, dwt=F32, acc=1, dw=0)),
    (STRIDE, dict(rows=0, dw=D + 2)), (ALIAS, dict(dw=A)), (ALIAS, dict(dw=B)), (ALIAS, dict(dw=C)),
    (STRIDE, dict(dw=D + 8)), (STRIDE, dict(dy=A + 2))])
def test_wgrad_refusals(sw, status, kw):
    assert wgrad(sw, **kw) == status


def test_timeout_flag_refuses_null(sw):
    assert sw.lib.swiglu_grouped_timeout_flag(None) == NULL


def test_python_layer_refuses_cpu_tensors_and_wrong_shapes(sw):
    x, w = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 32, 16).bfloat16()
    ends = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sw.swiglu_grouped_mm_fwd(x, w, ends)
    with pytest.raises(ValueError, match="CUDA"):
        sw.swiglu_grouped_mm_wgrad(x, x, ends)
    with pytest.raises(ValueError, match="CUDA"):
        sw.swiglu_ckpt8_fwd(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="even"):
        sw.swiglu_ckpt8_fwd(torch.zeros(4, 7))
    with pytest.raises(ValueError, match="save"):
        sw.swiglu_grouped_fc1_fwd(x, w, ends, save="fp4")
    with pytest.raises(ValueError, match="needs w"):
        sw.swiglu_ckpt8_bwd(torch.zeros(4, 8), torch.zeros(4, 16), torch.zeros(4, 2), dw=torch.zeros(4))


def limit(name):
    return int(re.search(rf"#define SWIGLU_GROUPED_{name} (\d+)\n", open(HEADER).read()).group(1))


@pytest.mark.parametrize("product", ["fc1", "fwd", "dgrad", "wgrad"])
def test_stated_limits_are_the_enforced_ones(sw, product):
    """The largest sizes that the header allows get as far as the check of pointers, the
    next ones do not."""
    def call(rows=16, groups=3, N=32, K=32, **kw):
        if product == "fc1":  # N counts gate and up rows
            return fc1(sw, x=0, rows=rows, groups=groups, n=N // 2, K=K)
        if product == "wgrad":
            return wgrad(sw, dy=0, rows=rows, groups=groups, N=N, K=K, **kw)
        return mm(sw, product, x=0, rows=rows, groups=groups, N=N, K=K)

    rows, features = limit("MAX_ROWS_WGRAD" if product == "wgrad" else "MAX_ROWS"), limit("MAX_FEATURES")
    assert call(rows=rows) == NULL and call(rows=rows + 1) == SHAPE
    assert call(K=features // 8 * 8) == NULL and call(K=features // 8 * 8 + 8) == SHAPE
    step = 16 if product == "fc1" else 8
    for groups in (1, 3, 8, 1024):
        N = features // groups // step * step
        assert call(groups=groups, N=N) == NULL and call(groups=groups, N=N + step) == SHAPE
    if product == "wgrad":
        for acc in (0, 1):
            assert call(rows=rows, dwt=F32, acc=acc) == NULL and call(rows=rows + 1, dwt=F32, acc=acc) == SHAPE


@pytest.mark.parametrize("missing", ["float8_e4m3fn", "float8_e8m0fnu"])
def test_a_torch_without_the_checkpoint_types_keeps_the_rest(sw, missing):
    """Such a torch imports the package; only the checkpoint's operators refuse."""
    import subprocess
    import sys

    code = f"""
import torch
del torch.{missing}
import gate_up_swiglu_gb300 as sw
import gate_up_swiglu_gb300.experts
x, w, ends = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 32, 16).bfloat16(), torch.zeros(2, dtype=torch.int32)
for fn in (lambda: sw.swiglu_gateup_fwd(x), lambda: sw.swiglu_grouped_fc1_fwd(x, w, ends, save="bf16"),
           lambda: sw.swiglu_grouped_mm_fwd(x, w, ends)):
    try:
        fn()
        assert False
    except ValueError as e:
        assert "CUDA" in str(e)
for fn in (lambda: sw.swiglu_ckpt8_fwd(x), lambda: sw.swiglu_ckpt8_bwd(x, x, x),
           lambda: sw.swiglu_grouped_fc1_fwd(x, w, ends, save="fp8")):
    try:
        fn()
        assert False
    except NotImplementedError as e:
        assert "float8" in str(e)
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]


def test_fc1_refuses_buffers_that_it_would_not_fill(sw):
    x, w, ends = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 32, 16).bfloat16(), torch.zeros(2, dtype=torch.int32)
    buf = torch.zeros(4, 32)
    for save, kw in ((None, dict(fc1=buf)), ("fp8", dict(fc1=buf)), (None, dict(q=buf)), (None, dict(scales=buf)),
                     ("bf16", dict(q=buf, scales=buf)), ("bf16", dict(scales=buf))):
        with pytest.raises(ValueError, match="is written with"):
            sw.swiglu_grouped_fc1_fwd(x, w, ends, save=save, **kw)
