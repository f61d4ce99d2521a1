"""The layer norm, forward and backward, against plain 64-bit implementations.

Tolerances.  u = 2^-24 is half a step of fp32.  A row's sums are trees of at most 16
terms in a thread, 5 levels in a warp and 32 warps: they are taken to be within
D u, D = 64, of the sums of absolute values.  So, with d = x - mean:
  mean:  D u mean|d| + u |mean|
  rstd:  relative D u / 2 + 4 u, and the mean's error squared over the variance (nothing)
  y:     |w| (D (|xhat| / 2 + mean|xhat|) + 8 |xhat|) u + 2 u (|xhat w| + |b|)
  dx:    rstd (D (mean|h| + |xhat| mean|h xhat|) + 8 (|h| + |c1| + |xhat c2|)) u
  dw, db: (rows / 19 + 100) u of the column's sum of absolute values: a group of rows
         after another in a chain, then up to 608 groups in 8 chains; the terms of dw
         carry 3 u of xhat
and half a step of the type that is stored."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U, D = 2.0 ** -24, 64
SHAPES = [(1, 1), (1, 2), (3, 7), (5, 16), (32, 256), (9, 100), (40, 257), (33, 512), (700, 384), (64, 1000), (17, 1024),
          (130, 2048), (20, 2047), (50, 4096), (9, 5503), (12, 8192), (6, 8200), (5, 12288), (3, 16384), (2, 16383),
          (4, 32768), (2, 40961), (3, 65536), (2, 70000), (5000, 64), (2500, 33)]


@pytest.fixture(scope="module")
def sw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(rows, n, dtype, pdtype=None, seed=0, pad=0, offset=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, n + pad) * 2 + offset).to(dtype)[:, :n]
    dy = r(rows, n + pad).to(dtype)[:, :n]
    pdtype = dtype if pdtype is None else pdtype
    return x, dy, (1 + 0.3 * r(n)).to(pdtype), (0.3 * r(n)).to(pdtype)


def fwd64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + torch.tensor(eps, dtype=F32).double()) ** -0.5
    xhat = d * rstd[:, None]
    w = torch.ones_like(xhat[0]) if w is None else w.double()
    b = torch.zeros_like(xhat[0]) if b is None else b.double()
    y = xhat * w + b
    off = w.abs() * (D * (xhat.abs() / 2 + xhat.abs().mean(1, keepdim=True)) + 8 * xhat.abs()) * U
    off = off + 2 * U * ((xhat * w).abs() + b.abs())
    return y, mean, rstd, off, D * U * d.abs().mean(1) + 2 * U * mean.abs()


def within(got, want, off, dtype, what):
    bad = ~((got.double() - want).abs() <= off + half_step(dtype) * (want.abs() + off) + 1e-38)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


def check_fwd(sw, x, w, b, eps=1e-5, **kw):
    y, mean, rstd = sw.swiglu_layer_norm_fwd(x, w, b, eps, return_stats=True, **kw)
    flat = x.reshape(-1, x.shape[-1])
    want, m, r, off, moff = fwd64(flat, w, b, eps)
    within(mean.reshape(-1), m, moff, F32, "mean")
    within(rstd.reshape(-1), r, (D / 2 + 4) * U * r, F32, "rstd")
    within(y.reshape(flat.shape), want, off, x.dtype, "y")
    return y, mean, rstd


def bwd64(dy, x, mean, rstd, w):
    dy, rstd = dy.double(), rstd.double()[:, None]
    xhat = (x.double() - mean.double()[:, None]) * rstd
    h = dy if w is None else dy * w.double()
    c1, c2 = h.mean(1, keepdim=True), (h * xhat).mean(1, keepdim=True)
    dx = rstd * (h - c1 - xhat * c2)
    off = D * (h.abs().mean(1, keepdim=True) + xhat.abs() * (h * xhat).abs().mean(1, keepdim=True))
    off = rstd * U * (off + 8 * (h.abs() + c1.abs() + (xhat * c2).abs()))
    k = (x.shape[0] / 19 + 100) * U
    t = (dy * xhat)
    return dx, t.sum(0), dy.sum(0), off, k * t.abs().sum(0), k * dy.abs().sum(0)


def check_bwd(sw, dy, x, w, bias_grad=True, eps=1e-5, pdtype=None, **kw):
    mean, rstd = sw.swiglu_layer_norm_fwd(x, None, None, eps, return_stats=True)[1:]
    dx, dw, db = sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, w, bias_grad, **kw)
    n = x.shape[-1]
    flat = lambda t: t.reshape(-1, n)  # noqa: E731
    want = bwd64(flat(dy), flat(x), mean.reshape(-1), rstd.reshape(-1), w)
    within(flat(dx), want[0], want[3], x.dtype, "dx")
    assert (dw is None) == (w is None) and (db is None) == (not bias_grad)
    if dw is not None:
        assert dw.dtype == w.dtype
        within(dw, want[1], want[4], dw.dtype, "dw")
    if db is not None:
        within(db, want[2], want[5], db.dtype, "db")
    return dx, dw, db


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward(sw, rows, n, dtype):
    x, _, w, b = make(rows, n, dtype)
    check_fwd(sw, x, w, b)


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward(sw, rows, n, dtype):
    x, dy, w, _ = make(rows, n, dtype, seed=1)
    check_bwd(sw, dy, x, w)


@pytest.mark.parametrize("n", [96, 200, 1024, 4096, 4099, 9000])
@pytest.mark.parametrize("pad", [0, 3, 8, 16])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_missing_parameters(sw, n, pad, dtype):
    x, dy, w, b = make(37, n, dtype, seed=2, pad=pad)
    check_fwd(sw, x, w, None)
    check_fwd(sw, x, None, None)
    check_fwd(sw, x, None, b)
    check_bwd(sw, dy, x, None, bias_grad=False)
    check_bwd(sw, dy, x, None, bias_grad=True)
    check_bwd(sw, dy, x, w, bias_grad=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,n", [(2600, 1), (2600, 6), (2600, 121), (2500, 250), (1300, 511), (700, 2043), (700, 4089),
                                    (700, 4096), (400, 8187), (330, 8190), (200, 12283), (90, 16379), (70, 32761),
                                    (40, 32767), (30, 65530), (700, 1020), (7, 9001), (17, 4001), (50, 8193), (33, 16389),
                                    (9, 20481)])
@pytest.mark.parametrize("widths,starts", [((0, 0, 0), (0, 0, 0)), ((11, 11, 11), (3, 3, 3)), ((3, 0, 0), (0, 0, 0)),
                                           ((16, 9, 10), (1, 6, 7)), ((2, 4, 16), (2, 1, 5)), ((8, 8, 8), (1, 1, 1))])
def test_rows_at_every_address(sw, rows, n, dtype, widths, starts):
    """Rows of any length, distance and start, x, dy and the results each its own; more rows
    than there are groups of threads; what lies around the results is left alone."""
    x, dy, w, b = make(rows, n, dtype, seed=n)
    hold = [torch.full((rows, n + k), 5.0, dtype=dtype, device="cuda") for k in widths]
    views = [t[:, min(k, t.shape[1] - n):][:, :n] for t, k in zip(hold, starts)]
    views[0].copy_(x)
    views[1].copy_(dy)
    x, dy, out = views

    def around():
        keep = torch.ones_like(hold[2], dtype=torch.bool)
        keep[:, out.storage_offset():out.storage_offset() + n] = False
        return bool((hold[2][keep] == 5).all())

    check_fwd(sw, x, w, b, y=out)
    assert around()
    check_bwd(sw, dy, x, w, dx=out)
    assert around()
    assert sw.layer_norm_timeout_flag() == 0


@pytest.mark.parametrize("rows,n", [(2600, 96), (2600, 97), (700, 4096), (700, 4091), (300, 8192), (200, 8199), (40, 16383),
                                    (40, 16384), (20, 30001), (20, 32768)])
def test_fp32_parameters_of_many_bf16_rows(sw, rows, n):
    x, dy, w, b = make(rows, n, BF16, F32, seed=9)
    check_fwd(sw, x, w, b)
    check_fwd(sw, x, None, b)
    dx, dw, db = check_bwd(sw, dy, x, w)
    assert dw.dtype == db.dtype == F32


@pytest.mark.parametrize("n", [64, 333, 4096, 20000])
def test_fp32_parameters_of_bf16_rows(sw, n):
    x, dy, w, b = make(41, n, BF16, F32, seed=3)
    check_fwd(sw, x, w, b)
    dx, dw, db = check_bwd(sw, dy, x, w)
    assert dw.dtype == db.dtype == F32


@pytest.mark.parametrize("dtype,offset", [(F32, 1e4), (F32, -3e5), (BF16, 200.0)])
@pytest.mark.parametrize("n", [300, 4096, 40000])
def test_far_mean(sw, dtype, offset, n):
    x, dy, w, b = make(11, n, dtype, seed=4, offset=offset)
    check_fwd(sw, x, w, b)
    check_bwd(sw, dy, x, w)


def test_three_dimensions_misaligned_and_given_outputs(sw):
    x, dy, w, b = make(30, 256, BF16, seed=5)
    check_fwd(sw, x.view(5, 6, 256), w, b)
    check_bwd(sw, dy.view(5, 6, 256), x.view(5, 6, 256), w)
    buf = torch.full((30, 300), 5.0, dtype=BF16, device="cuda")
    check_fwd(sw, x, w, b, y=buf[:, 1:257])
    assert bool((buf[:, 0] == 5).all()) and bool((buf[:, 257:] == 5).all())
    dxb = torch.full((30, 300), 5.0, dtype=BF16, device="cuda")
    check_bwd(sw, dy, x, w, dx=dxb[:, 7:263])
    assert bool((dxb[:, :7] == 5).all()) and bool((dxb[:, 263:] == 5).all())
    wm = torch.cat([w, w])[1:257]  # parameters at an odd address
    check_fwd(sw, x, wm, None)
    check_bwd(sw, dy, x, wm)


@pytest.mark.parametrize("n", [128, 1000, 9000, 70000])
def test_nan_and_infinity_stay_in_their_row(sw, n):
    x, dy, w, b = make(6, n, F32, seed=6)
    x[1, n // 2], x[4, 0] = float("nan"), float("inf")
    y, mean, rstd = sw.swiglu_layer_norm_fwd(x, w, b, return_stats=True)
    bad = torch.tensor([False, True, False, False, True, False], device="cuda")
    for t in (y, mean[:, None], rstd[:, None]):
        assert torch.equal((~torch.isfinite(t)).any(1), bad)
    dx, dw, db = sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, w)
    assert torch.equal(torch.isnan(dx).all(1), bad) and torch.equal(torch.isnan(dx).any(1), bad)
    assert bool(torch.isfinite(db).all())


def test_constant_rows_and_eps(sw):
    x = torch.full((4, 500), 3.0, device="cuda")
    for eps in (1e-5, 1e-12, 0.25):
        y, mean, rstd = sw.swiglu_layer_norm_fwd(x, eps=eps, return_stats=True)
        assert bool((y == 0).all()) and bool((mean == 3).all())
        assert torch.allclose(rstd, torch.full_like(rstd, eps ** -0.5), rtol=1e-6)
    x, _, w, b = make(8, 640, F32, seed=7)
    check_fwd(sw, x, w, b, eps=0.5)


def test_empty(sw):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    assert sw.swiglu_layer_norm_fwd(e(0, 64), e(64)).shape == (0, 64)
    assert sw.swiglu_layer_norm_fwd(e(3, 0)).shape == (3, 0)
    dx, dw, db = sw.swiglu_layer_norm_bwd(e(0, 64), e(0, 64), e(0), e(0), torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("rows,n,dtype", [(4000, 4096, BF16), (3000, 5503, F32), (20000, 256, BF16)])
def test_same_bits_every_time(sw, rows, n, dtype):
    x, dy, w, _ = make(rows, n, dtype, seed=8)
    one, two = (check_bwd(sw, dy, x, w) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_streams_and_graphs(sw):
    """A call on another stream; one workspace for captured calls that follow each other,
    replayed on new inputs."""
    x, dy, w, b = make(300, 1024, BF16, seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = sw.swiglu_layer_norm_fwd(x, w, b, stream=s)
    s.synchronize()
    assert torch.equal(y, sw.swiglu_layer_norm_fwd(x, w, b))
    ws = torch.empty(sw.layer_norm_bwd_workspace_bytes(300, 1024), dtype=torch.uint8, device="cuda")
    mean, rstd = sw.swiglu_layer_norm_fwd(x, return_stats=True)[1:]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sw.swiglu_layer_norm_fwd(x, w, b, y=y, mean=mean, rstd=rstd)
        first = sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, w, workspace=ws)
        second = sw.swiglu_layer_norm_bwd(x, x, mean, rstd, w, workspace=ws)
    for seed in (10, 11):
        nx, ndy, _, _ = make(300, 1024, BF16, seed=seed)
        x.copy_(nx), dy.copy_(ndy)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in ((first, sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, w)),
                          (second, sw.swiglu_layer_norm_bwd(x, x, mean, rstd, w))):
            assert all(torch.equal(a, c) for a, c in zip(got, want))
        check_fwd(sw, x, w, b)


@pytest.mark.parametrize("rows,n,dtype", [(700, 8193, BF16), (500, 12296, BF16), (301, 20000, F32), (90, 32768, F32),
                                          (613, 16384, BF16), (1, 9000, F32), (2, 30001, BF16)])
def test_rows_split_over_a_cluster(sw, rows, n, dtype):
    """Many rows through each group of a cluster, and fewer than there are groups."""
    x, dy, w, b = make(rows, n, dtype, seed=12)
    check_fwd(sw, x, w, b)
    first = check_bwd(sw, dy, x, w)
    assert all(torch.equal(a, c) for a, c in zip(first, check_bwd(sw, dy, x, w)))
    assert sw.layer_norm_timeout_flag() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("rows,n", [(6, 40), (6, 500), (6, 512), (700, 513), (700, 4000), (700, 4095), (700, 4096),
                                    (6, 5503), (90, 8193), (40, 20000), (40, 32761), (40, 32768), (3, 70000)])
def test_backward_of_constant_rows_of_large_values(sw, rows, n, pad, dtype):
    """xhat = 0, and dx = rstd (h - mean(h)), whether or not the threads that share a row have
    columns past its end (mean * rstd is beyond fp32)."""
    _, dy, w, _ = make(rows, n, dtype, seed=n, pad=pad)
    x = torch.full((rows, n + pad), 1e33, device="cuda").to(dtype)[:, :n]
    mean, rstd = x[:, 0].float().contiguous(), torch.full((rows,), 1e6, device="cuda")
    dx, dw, db = sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, w)
    want = bwd64(dy, x, mean, rstd, w)
    within(dx, want[0], want[3], dtype, "dx")
    assert bool((dw == 0).all())
    within(db, want[2], want[5], dtype, "db")


@pytest.mark.parametrize("rows,n,dtype", [(3000, 155651, F32), (3000, 155652, F32), (600, 700009, BF16), (600, 700008, BF16)])
def test_column_sums_of_many_very_long_rows(sw, rows, n, dtype):
    """Equal terms, whose rounding errors do not cancel: a chain over 3000 rows would be some
    500 units off, segments are within the bound of every other length."""
    terms = torch.tensor([0.1, 0.3, 0.7, 1.1, 1.3, 0.013], device="cuda")[torch.arange(n, device="cuda") % 6].to(dtype)
    dy, x = terms.repeat(rows, 1), torch.ones(1, n, device="cuda", dtype=dtype).repeat(rows, 1)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx, dw, db = sw.swiglu_layer_norm_bwd(dy, x, mean, rstd, torch.ones(n, device="cuda"), dx=torch.empty_like(x))
    want = rows * terms.double()
    for got in (dw, db):
        within(got, want, (rows / 19 + 100) * U * want, F32, "sums")
    h = terms.double()
    c1, c2 = h.mean(), h.mean()  # xhat = 1
    off = U * (D * (h.abs().mean() + h.abs().mean()) + 8 * (h.abs() + c1.abs() + c2.abs()))
    for r in (0, 255, 256, rows - 1):
        within(dx[r], h - c1 - c2, off, dtype, "dx")
