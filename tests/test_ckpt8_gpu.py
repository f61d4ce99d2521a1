"""The 8-bit activation checkpoint against plain 64-bit implementations.

Tolerances (fixed before the first run):
  * codes and scales: equal (the format is exact arithmetic; NaN meets NaN);
  * y of the forward: bit for bit that of swiglu_gateup_fwd / _weighted_fwd;
  * dx and y of the backward: helpers.mismatches' rules at the restored x;
  * dw: an fp32 sum shared by at least the 32 lanes of a warp has chains of at
    most n / 32 + 16 additions, each 2^-24 relative, plus the error of the terms
    (2^-17 for bf16's hardware exponential and reciprocal, 2e-6 or 1e-7 each for
    fp32) and one step of fp32.
"""
import math

import pytest
import torch

import moe_reference as R
from helpers import assert_bitwise, assert_parity

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


def _x(rows, n, dt, seed, std=4.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, 2 * n, generator=g) * std).to(DT[dt])


def _guarded(rows, cols, stride, dtype, lead=3):
    """A [rows, cols] view with the given row stride inside a patterned buffer."""
    buf = torch.full((lead * stride + rows * stride + 64,), 0x5a, dtype=torch.uint8, device="cuda")
    if dtype.itemsize > 1:
        buf = torch.full((lead * stride + rows * stride + 64,), 0x5a5a if dtype.itemsize == 2 else 0x5a5a5a5a,
                         dtype=torch.int16 if dtype.itemsize == 2 else torch.int32, device="cuda")
    view = buf.view(dtype)[lead * stride:lead * stride + rows * stride].view(rows, stride)[:, :cols]
    return buf, view


def _untouched(buf, rows, cols, stride, lead=3):
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[lead * stride:lead * stride + rows * stride].view(rows, stride)[:, :cols] = False
    pat = {1: 0x5a, 2: 0x5a5a, 4: 0x5a5a5a5a}[buf.element_size()]
    return bool((buf[keep] == pat).all())


def _check_codes(q, scales, x, what):
    qr, cr = R.checkpoint(x)
    assert torch.equal(scales.view(torch.uint8).cpu().long(), cr), f"{what}: scales differ"
    qv = q.cpu().float().double()
    same = (qv == qr) | (qv.isnan() & qr.isnan())
    assert bool(same.all()), f"{what}: {int((~same).sum())} codes differ, first {(~same).nonzero()[:4].tolist()}"


SHAPES = [(1, 1), (1, 8), (3, 31), (3, 32), (5, 33), (2, 40), (7, 64), (4, 72), (33, 256), (9, 517), (16, 1000),
          (3, 4096), (2, 5503)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_forward(sw, rows, n, dt, weighted):
    x = _x(rows, n, dt, rows * 1000 + n)
    w = torch.rand(rows, generator=torch.Generator().manual_seed(n)).cuda() if weighted else None
    xd = x.cuda()
    y, q, scales = sw.swiglu_ckpt8_fwd(xd, w)
    assert_bitwise(y, sw.swiglu_gateup_weighted_fwd(xd, w) if weighted else sw.swiglu_gateup_fwd(xd), "y")
    _check_codes(q, scales, x, f"{dt} {rows}x{n}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_backward(sw, rows, n, dt, weighted):
    x = _x(rows, n, dt, rows * 1000 + n + 1, std=2.0)
    g = torch.Generator().manual_seed(n + 7)
    dy = torch.randn(rows, n, generator=g).to(DT[dt])
    w = torch.rand(rows, generator=g) if weighted else None
    _, q, scales = sw.swiglu_ckpt8_fwd(x.cuda())
    dx, dw, y = sw.swiglu_ckpt8_bwd(dy.cuda(), q, scales, None if w is None else w.cuda(), return_y=True)
    xr = R.restored(q.cpu(), scales.cpu())
    rdx, rdw, ry, rabs = R.swiglu_bwd(dy, xr, w)
    assert_parity(dx, rdx.to(DT[dt]), "dx")
    assert_parity(y, ry.to(DT[dt]), "y")
    dx2, _, none = sw.swiglu_ckpt8_bwd(dy.cuda(), q, scales, None if w is None else w.cuda())
    assert none is None
    assert_bitwise(dx2, dx, "dx must not depend on y being asked for")
    if weighted:
        tol = (n / 32 + 16) * 2.0 ** -24 * rabs + 2.0 ** -23 * rdw.abs()
        tol += 2.0 ** -17 * rabs if dt == "bf16" else 2e-6 * rabs + n * 1e-7
        assert bool(((dw.cpu().double() - rdw).abs() <= tol).all())
    else:
        assert dw is None


def test_gradient_against_differences(sw):
    """dx and dw are the slopes of sum(dy * y) at the restored x (central differences in float64)."""
    rows, n = 3, 40
    x = _x(rows, n, "f32", 5, std=1.0)
    g = torch.Generator().manual_seed(6)
    dy, w = torch.randn(rows, n, generator=g), torch.rand(rows, generator=g) + 0.5
    _, q, scales = sw.swiglu_ckpt8_fwd(x.cuda())
    dx, dw, _ = sw.swiglu_ckpt8_bwd(dy.cuda(), q, scales, w.cuda())
    xr = R.restored(q.cpu(), scales.cpu())

    def loss(x, w):
        return (dy.double() * w[:, None] * R.silu64(x[:, :n]) * x[:, n:]).sum()

    h = 1e-5
    for k in torch.randint(0, rows * 2 * n, (40,), generator=g).tolist():
        e = torch.zeros(rows * 2 * n, dtype=torch.float64)
        e[k] = h
        e = e.view(rows, 2 * n)
        slope = (loss(xr + e, w.double()) - loss(xr - e, w.double())) / (2 * h)
        assert abs(float(dx.view(-1)[k]) - float(slope)) <= 1e-6 + 4e-6 * abs(float(slope))
    for r in range(rows):
        e = torch.zeros(rows, dtype=torch.float64)
        e[r] = h
        slope = (loss(xr, w.double() + e) - loss(xr, w.double() - e)) / (2 * h)
        assert abs(float(dw[r]) - float(slope)) <= 1e-5 + 1e-5 * abs(float(slope))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [32, 45, 64, 96])
def test_special_values(sw, n, dt):
    """Zeros, subnormals, block maxima around 448 * 2^k, the type's largest and
    lowest values, infinities and NaN, each in blocks with and without company."""
    big = float(torch.finfo(DT[dt]).max)
    tiny = float(torch.finfo(DT[dt]).smallest_normal)
    cols = [0.0, -0.0, tiny, -tiny / 64, 448.0, 449.0, 450.0, 464.0, 1.75, 1.7578125, 3.5, -3.515625, big, -big,
            float("inf"), float("-inf"), float("nan"), 1e-30, 2.0 ** -127, 2.0 ** -133, 1.0, 0.0625, 0.001953125]
    rows = []
    for i, v in enumerate(cols):
        alone = torch.zeros(2 * n)
        alone[i % n] = v
        alone[n + (3 * i) % n] = v
        rows.append(alone)
        rows.append(torch.where(torch.arange(2 * n) % 7 == i % 7, torch.tensor(v), torch.randn(
            2 * n, generator=torch.Generator().manual_seed(i))))
    x = torch.stack(rows).to(DT[dt])
    xd = x.cuda()
    y, q, scales = sw.swiglu_ckpt8_fwd(xd)
    _check_codes(q, scales, x, f"special {dt} n {n}")
    assert_bitwise(torch.nan_to_num(y, 1.0), torch.nan_to_num(sw.swiglu_gateup_fwd(xd), 1.0), "y")
    dy = torch.randn(x.shape[0], n, generator=torch.Generator().manual_seed(1)).to(DT[dt])
    dx, _, y2 = sw.swiglu_ckpt8_bwd(dy.cuda(), q, scales, return_y=True)
    rdx, _, ry, _ = R.swiglu_bwd(dy, R.restored(q.cpu(), scales.cpu()))
    # rows whose 64-bit result leaves the type's range are not compared: big * big
    fine = torch.cat([rdx, ry], 1).abs().nan_to_num(0.0).amax(1) < big / 4
    assert_parity(dx.cpu()[fine], rdx.to(DT[dt])[fine], "dx")
    assert_parity(y2.cpu()[fine], ry.to(DT[dt])[fine], "y")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_every_code_restores(sw, dt):
    """The backward at all 256 codes as gates under several scales (deep tails
    among them: gates far below -64)."""
    q = torch.arange(256, dtype=torch.uint8).view(8, 32)
    q = torch.cat([q, torch.full((8, 32), 0x38, dtype=torch.uint8)], 1)  # up = 1
    for code in (0, 100, 120, 127, 128, 131, 140):
        scales = torch.tensor([[code, 127]], dtype=torch.uint8).repeat(8, 1).view(torch.float8_e8m0fnu)
        qf = q.view(torch.float8_e4m3fn)
        dy = torch.ones(8, 32, dtype=DT[dt])
        dx, _, y = sw.swiglu_ckpt8_bwd(dy.cuda(), qf.cuda(), scales.cuda(), return_y=True)
        rdx, _, ry, _ = R.swiglu_bwd(dy, R.restored(qf, scales))
        assert_parity(dx, rdx.to(DT[dt]), f"dx, scale code {code}")
        assert_parity(y, ry.to(DT[dt]), f"y, scale code {code}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,pads", [(64, (16, 16, 32, 4)), (64, (1, 3, 5, 1)), (40, (8, 8, 8, 0)), (33, (0, 2, 1, 7)),
                                    (256, (8, 24, 16, 2))])
def test_strides_and_guards(sw, n, pads, dt):
    """Rows inside wider buffers; nothing outside the rows is written."""
    rows, (px, py, pq, ps) = 11, pads
    nb = -(-n // 32)
    x = _x(rows, n, dt, n)
    bx, xv = _guarded(rows, 2 * n, 2 * n + px, DT[dt])
    xv.copy_(x)
    by, yv = _guarded(rows, n, n + py, DT[dt])
    bq, qv = _guarded(rows, 2 * n, 2 * n + pq, torch.float8_e4m3fn)
    bs, sv = _guarded(rows, 2 * nb, 2 * nb + ps, torch.float8_e8m0fnu)
    y, q, scales = sw.swiglu_ckpt8_fwd(xv, None, yv, qv, sv)
    assert y is yv and q is qv and scales is sv
    assert_bitwise(yv, sw.swiglu_gateup_fwd(x.cuda()), "y")
    _check_codes(qv, sv, x, "strided")
    assert _untouched(by, rows, n, n + py) and _untouched(bq, rows, 2 * n, 2 * n + pq)
    assert _untouched(bs, rows, 2 * nb, 2 * nb + ps)
    w = torch.rand(rows, generator=torch.Generator().manual_seed(2)).cuda()
    dy = torch.randn(rows, n, generator=torch.Generator().manual_seed(3)).to(DT[dt]).cuda()
    bd, dyv = _guarded(rows, n, n + py, DT[dt])
    dyv.copy_(dy)
    bdx, dxv = _guarded(rows, 2 * n, 2 * n + px, DT[dt])
    by2, y2v = _guarded(rows, n, n + py, DT[dt])
    sw.swiglu_ckpt8_bwd(dyv, qv, sv, w, dx=dxv, y=y2v)
    xr = R.restored(qv.cpu(), sv.cpu())
    rdx, _, ry, _ = R.swiglu_bwd(dy.cpu(), xr, w.cpu())
    assert_parity(dxv, rdx.to(DT[dt]), "dx")
    assert_parity(y2v, ry.to(DT[dt]), "y")
    assert _untouched(bdx, rows, 2 * n, 2 * n + px) and _untouched(by2, rows, n, n + py)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 4, 34, 36, 62, 66, 68, 100, 126, 250, 252, 260, 1030, 2730, 5460])
def test_narrow_packs(sw, n, dt):
    """Widths of packs of 8 and 4 bytes; from an odd column on, of single elements: the
    same codes and bits either way, with values of every care in some rows."""
    rows = 9
    x = _x(rows, n, dt, 31 * n, std=2.0)
    x[1, 0], x[2, n], x[3, n - 1], x[4, 2 * n - 1], x[5, n // 2] = math.inf, -math.inf, math.nan, 3e38, -90.0
    x[6] = 0.0
    w = torch.rand(rows, generator=torch.Generator().manual_seed(n)).cuda()
    dy = torch.randn(rows, n, generator=torch.Generator().manual_seed(n + 1)).to(DT[dt])
    results = []
    for off in (0, 1):
        xv = torch.zeros(rows, 2 * n + 8, dtype=DT[dt], device="cuda")[:, off:off + 2 * n]
        xv.copy_(x)
        dyv = torch.zeros(rows, n + 8, dtype=DT[dt], device="cuda")[:, off:off + n]
        dyv.copy_(dy)
        y, q, scales = sw.swiglu_ckpt8_fwd(xv, w)
        _check_codes(q, scales, x, f"{dt} n {n} from column {off}")
        assert_bitwise(y, sw.swiglu_gateup_weighted_fwd(x.cuda(), w), "y")
        plain = sw.swiglu_ckpt8_bwd(dyv, q, scales, None, return_y=True)
        weighted = sw.swiglu_ckpt8_bwd(dyv, q, scales, w, return_y=True)
        results.append((q.view(torch.uint8), plain[0], plain[2], weighted[0], weighted[2]))
        usual = [0, 5, 6, 7, 8]
        xr = R.restored(q.cpu(), scales.cpu())[usual]
        rdx, rdw, ry, rabs = R.swiglu_bwd(dy[usual], xr, w.cpu()[usual])
        assert_parity(weighted[0][usual], rdx.to(DT[dt]), "dx")
        assert_parity(weighted[2][usual], ry.to(DT[dt]), "y")
        tol = (n / 32 + 16) * 2.0 ** -24 * rabs + 2.0 ** -23 * rdw.abs()
        tol += 2.0 ** -17 * rabs if dt == "bf16" else 2e-6 * rabs + n * 1e-7
        assert bool(((weighted[1].cpu().double()[usual] - rdw).abs() <= tol).all()), "dw"
    for a, b in zip(*results):
        if a.dtype == torch.uint8:
            assert torch.equal(a, b)
        else:
            nan = a.isnan()
            assert torch.equal(nan, b.isnan()) and torch.equal(a[~nan], b[~nan])


def test_three_dimensions_streams_and_repeats(sw):
    x = _x(24, 96, "bf16", 9).cuda().view(6, 4, 192)
    w = torch.rand(24, device="cuda")
    dy = torch.randn(6, 4, 96, device="cuda").bfloat16()
    y, q, s = sw.swiglu_ckpt8_fwd(x, w)
    assert y.shape == (6, 4, 96) and q.shape == (6, 4, 192) and s.shape == (6, 4, 6)
    dx, dw, y2 = sw.swiglu_ckpt8_bwd(dy, q, s, w, return_y=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = sw.swiglu_ckpt8_fwd(x, w)
        back = sw.swiglu_ckpt8_bwd(dy, again[1], again[2], w, return_y=True)
    third = sw.swiglu_ckpt8_bwd(dy, q, s, w, return_y=True, stream=side)
    torch.cuda.synchronize()
    for a, b in zip((y, dx, dw, y2, dx, dw, y2), (again[0], *back, *third)):
        assert torch.equal(a, b)
    assert torch.equal(q.view(torch.uint8), again[1].view(torch.uint8))


def test_empty(sw):
    x = torch.empty(0, 64, device="cuda")
    y, q, s = sw.swiglu_ckpt8_fwd(x)
    assert y.shape == (0, 32) and q.shape == (0, 64) and s.shape == (0, 2)
    dx, dw, _ = sw.swiglu_ckpt8_bwd(torch.empty(0, 32, device="cuda"), q, s, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and dw.shape == (0,)
    dw = torch.full((5,), 3.0, device="cuda")
    _, q, s = sw.swiglu_ckpt8_fwd(torch.empty(5, 0, device="cuda"))
    sw.swiglu_ckpt8_bwd(torch.empty(5, 0, device="cuda"), q, s, torch.ones(5, device="cuda"), dw=dw)
    assert float(dw.abs().max()) == 0.0


def test_graph_capture(sw):
    x = _x(64, 128, "bf16", 3).cuda()
    dy = torch.randn(64, 128, device="cuda").bfloat16()
    w = torch.rand(64, device="cuda")
    sw.swiglu_ckpt8_bwd(dy, *sw.swiglu_ckpt8_fwd(x, w)[1:], w, return_y=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, q, s = sw.swiglu_ckpt8_fwd(x, w)
        dx, dw, y2 = sw.swiglu_ckpt8_bwd(dy, q, s, w, return_y=True)
    x.copy_(_x(64, 128, "bf16", 4))
    graph.replay()
    torch.cuda.synchronize()
    ey, eq, es = sw.swiglu_ckpt8_fwd(x, w)
    edx, edw, ey2 = sw.swiglu_ckpt8_bwd(dy, eq, es, w, return_y=True)
    for a, b in ((y, ey), (dx, edx), (dw, edw), (y2, ey2), (q.view(torch.uint8), eq.view(torch.uint8))):
        assert torch.equal(a, b)


def test_large_offsets(sw):
    """Element offsets past 2^31 in x and dx, and past 2^32 bytes: sampled rows."""
    rows, n = 70001, 16384  # x: 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, 2 * n, dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, 8192):
        x[at:at + 8192] = torch.randn(x[at:at + 8192].shape, generator=g, device="cuda")
    w = torch.rand(rows, generator=g, device="cuda")
    y, q, s = sw.swiglu_ckpt8_fwd(x, w)
    pick = torch.tensor([0, 1, 32767, 32768, 65535, 65536, 70000])
    _check_codes(q[pick.cuda()], s[pick.cuda()], x[pick.cuda()].cpu(), "large")
    dy = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
    dx, dw, y2 = sw.swiglu_ckpt8_bwd(dy, q, s, w, return_y=True)
    rdx, rdw, ry, rabs = R.swiglu_bwd(dy[pick.cuda()].cpu(), R.restored(q[pick.cuda()].cpu(), s[pick.cuda()].cpu()),
                                      w[pick.cuda()].cpu())
    assert_parity(dx[pick.cuda()], rdx.bfloat16(), "dx")
    assert_parity(y2[pick.cuda()], ry.bfloat16(), "y")
    tol = (n / 32 + 16) * 2.0 ** -24 * rabs + 2.0 ** -23 * rdw.abs() + 2.0 ** -17 * rabs
    assert bool(((dw[pick.cuda()].cpu().double() - rdw).abs() <= tol).all())


def test_python_layer_refusals(sw):
    x = torch.zeros(4, 64, device="cuda")
    y, q, s = sw.swiglu_ckpt8_fwd(x)
    w = torch.ones(4, device="cuda")
    dy = torch.zeros(4, 32, device="cuda")
    for bad in (lambda: sw.swiglu_ckpt8_fwd(x.half()), lambda: sw.swiglu_ckpt8_fwd(x, w[:3]),
                lambda: sw.swiglu_ckpt8_fwd(x, w.double()), lambda: sw.swiglu_ckpt8_fwd(x, w.cpu()),
                lambda: sw.swiglu_ckpt8_fwd(x[:, ::2]), lambda: sw.swiglu_ckpt8_fwd(x, None, y.bfloat16()),
                lambda: sw.swiglu_ckpt8_fwd(x, None, y[:3]), lambda: sw.swiglu_ckpt8_fwd(x, None, None, q.view(torch.uint8)),
                lambda: sw.swiglu_ckpt8_fwd(x, None, None, q, s[:, :1]), lambda: sw.swiglu_ckpt8_bwd(dy, q.view(torch.uint8), s),
                lambda: sw.swiglu_ckpt8_bwd(dy, q[:3], s), lambda: sw.swiglu_ckpt8_bwd(dy, q, s[:, :1]),
                lambda: sw.swiglu_ckpt8_bwd(dy[:, :31], q, s), lambda: sw.swiglu_ckpt8_bwd(dy, q, s, w[:2]),
                lambda: sw.swiglu_ckpt8_bwd(dy, q, s, dw=w), lambda: sw.swiglu_ckpt8_bwd(dy, q.cpu(), s),
                lambda: sw.swiglu_ckpt8_bwd(dy, q, s, w, y=dy.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sw.SwigluError, match="ALIAS"):
        sw.swiglu_ckpt8_bwd(dy, q, s, y=dy)
