"""The experts' grouped products against plain 64-bit implementations.

Tolerances (fixed before the first run):
  * integer inputs: every product and partial sum is exact in fp32, so results
    equal the exact value rounded once, bit for bit (y of the first product:
    one bf16 step, it passes through the exponential);
  * other inputs: the tensor cores add with truncation, at most 2^-23 relative of
    the running sum per addition, so a sum of D terms is within D 2^-23 sum|t| of
    the exact one; plus one bf16 step where it is rounded to bf16.  fp32 weight
    gradients are summed in segments of 4096 rows.
"""
import math

import pytest
import torch

import moe_reference as R
from helpers import bf16_ordered

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    yield sw
    assert sw.grouped_timeout_flag() == 0


def _ints(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ends(counts):
    return torch.tensor(counts, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


# (rows per expert, rows of no expert)
GROUPS = [([1], 0), ([0, 1], 0), ([1, 0, 0, 1], 1), ([0, 0], 3), ([31, 32, 33], 0), ([63, 64, 65], 2),
          ([255, 0, 256, 257], 0), ([300, 1, 513, 0, 7], 40), ([5] * 40, 0), ([1100, 20], 0)]
# the widest give enough tiles for the kernel of CTA pairs, the others split the depth
WIDTHS = [(8, 8), (64, 64), (136, 72), (256, 200), (264, 520), (4104, 72), (72, 4104), (2056, 2176)]


def _same_bits(a, b):
    return torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a.view(torch.int32),
                       b.view(torch.int16) if b.dtype == torch.bfloat16 else b.view(torch.int32))


@pytest.mark.parametrize("counts,tail", GROUPS)
@pytest.mark.parametrize("N,K", WIDTHS)
def test_products_exact_on_integers(sw, counts, tail, N, K):
    """Any misplaced row, column, group or zero shows: forward, both gradients."""
    g = _gen(sum(counts) * 31 + N + K)
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w, dy = _ints(g, rows, K), _ints(g, E, N, K), _ints(g, rows, N)
    y = sw.swiglu_grouped_mm_fwd(x, w, ends)
    assert _same_bits(y + 0.0, R.mm(x, w, ends)[0].bfloat16() + 0.0)
    dx = sw.swiglu_grouped_mm_dgrad(dy, w, ends)
    assert _same_bits(dx + 0.0, R.dgrad(dy, w, ends)[0].bfloat16() + 0.0)
    ref = R.wgrad(dy, x, ends, E)[0]
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends)
    assert _same_bits(dw + 0.0, ref.bfloat16() + 0.0)
    dw32 = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32)
    assert _same_bits(dw32 + 0.0, ref.float() + 0.0)
    more = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=dw32.clone(), accumulate=True)
    assert _same_bits(more + 0.0, (2 * ref).float() + 0.0)


@pytest.mark.parametrize("counts,tail", GROUPS)
@pytest.mark.parametrize("n,K", [(8, 8), (24, 64), (72, 136), (128, 64), (200, 264), (160, 72), (2056, 136),
                                 (40, 2056)])
@pytest.mark.parametrize("probs", [False, True])
def test_first_product_exact_on_integers(sw, counts, tail, n, K, probs):
    """fc1 and its checkpoint bit for bit, y within one bf16 step."""
    g = _gen(sum(counts) * 17 + n + K)
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w = _ints(g, rows, K, top=1), _ints(g, E, 2 * n, K, top=2)
    p = torch.rand(rows, generator=g, device="cuda") if probs else None
    ref = R.mm(x, w, ends)[0]
    y64 = R.silu64(ref[:, :n]) * ref[:, n:]
    if probs:
        y64 = y64 * p.double()[:, None]
    y = sw.swiglu_grouped_fc1_fwd(x, w, ends, p)
    assert int((bf16_ordered(y) - bf16_ordered(y64.bfloat16())).abs().max()) <= 1
    y2, fc1 = sw.swiglu_grouped_fc1_fwd(x, w, ends, p, save="bf16")
    y3, q, scales = sw.swiglu_grouped_fc1_fwd(x, w, ends, p, save="fp8")
    assert _same_bits(y2, y) and _same_bits(y3, y)
    assert _same_bits(fc1 + 0.0, ref.bfloat16() + 0.0)
    qr, cr = R.checkpoint(ref)
    assert torch.equal(scales.view(torch.uint8).long(), cr)
    assert torch.equal(q.float().double(), qr)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def _step(v):
    return v.abs().clamp(min=2.0 ** -126) * 2.0 ** -7


@pytest.mark.parametrize("counts,tail,N,K", [([700, 0, 33, 1200], 11, 520, 1416), ([3, 1, 0, 2], 0, 1160, 2048),
                                             ([200] * 9, 0, 328, 96)])
def test_products_on_normals(sw, counts, tail, N, K):
    g = _gen(N * K)
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w, dy = _normal(g, rows, K), _normal(g, E, N, K, std=K ** -0.5), _normal(g, rows, N)
    for got, (ref, a), depth in ((sw.swiglu_grouped_mm_fwd(x, w, ends), R.mm(x, w, ends), K),
                                 (sw.swiglu_grouped_mm_dgrad(dy, w, ends), R.dgrad(dy, w, ends), N),
                                 (sw.swiglu_grouped_mm_wgrad(dy, x, ends), R.wgrad(dy, x, ends, E), max(counts))):
        assert bool(((got.double() - ref).abs() <= _step(ref) + depth * 2.0 ** -23 * a).all())
    ref, a = R.wgrad(dy, x, ends, E)
    got = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32)
    assert bool(((got.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + max(counts) * 2.0 ** -23 * a).all())


@pytest.mark.parametrize("counts,tail,n,K", [([700, 0, 33, 1200], 11, 264, 1416), ([3, 1, 0, 2], 0, 584, 2048)])
def test_first_product_on_normals(sw, counts, tail, n, K):
    g = _gen(n * K)
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w, p = _normal(g, rows, K), _normal(g, E, 2 * n, K, std=4 * K ** -0.5), torch.rand(rows, generator=g,
                                                                                       device="cuda")
    y, fc1 = sw.swiglu_grouped_fc1_fwd(x, w, ends, p, save="bf16")
    ref, a = R.mm(x, w, ends)
    gam = K * 2.0 ** -23
    assert bool(((fc1.double() - ref).abs() <= _step(ref) + gam * a).all())
    gt, u, ag, au = ref[:, :n], ref[:, n:], gam * a[:, :n], gam * a[:, n:]
    y64 = R.silu64(gt) * u * p.double()[:, None]
    # |silu'| <= 1.1; the activation's own error is far inside the bf16 step
    tol = _step(y64) + p.double()[:, None] * (1.1 * ag * u.abs() + R.silu64(gt).abs() * au + 1.1 * ag * au)
    assert bool(((y.double() - y64).abs() <= tol).all())
    # the checkpoint holds the product: restored within half an e4m3 step of the
    # block's scale (values below it: half of 2^-9 of the scale), and the sums' error
    _, q, scales = sw.swiglu_grouped_fc1_fwd(x, w, ends, p, save="fp8")
    back = R.restored(q, scales)
    nb = scales.shape[1] // 2
    f = torch.exp2(scales.view(torch.uint8).double() - 127).view(rows, 2, nb)
    f = f[:, :, torch.arange(n, device="cuda") // 32].reshape(rows, 2 * n)
    assert bool(((back - ref).abs() <= ref.abs() * 2.0 ** -4 + f * 2.0 ** -10 + gam * a).all())


def test_any_ends_are_safe(sw):
    """Values out of order, negative or past the rows: the running maximum within [0, rows]."""
    g = _gen(3)
    rows, E, N, K = 200, 6, 72, 136
    x, w, dy = _ints(g, rows, K), _ints(g, E, N, K), _ints(g, rows, N)
    for vals in ([-5, 30, 10, 90, 2 ** 31 - 1, 7], [0] * 6, [-2 ** 31] * 6, [200] * 6, [199, 0, 0, 0, 0, 0],
                 [500, 20, 30, 40, 50, 60], [10, 20, 30, 40, 50, 60]):
        ends = torch.tensor(vals, dtype=torch.int32, device="cuda")
        assert _same_bits(sw.swiglu_grouped_mm_fwd(x, w, ends) + 0.0, R.mm(x, w, ends)[0].bfloat16() + 0.0)
        assert _same_bits(sw.swiglu_grouped_mm_dgrad(dy, w, ends) + 0.0, R.dgrad(dy, w, ends)[0].bfloat16() + 0.0)
        assert _same_bits(sw.swiglu_grouped_mm_wgrad(dy, x, ends) + 0.0, R.wgrad(dy, x, ends, E)[0].bfloat16() + 0.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_stays_in_its_row_and_group(sw, bad):
    """Rows of NaN or infinity: no other row, no other group's dW, and rows of no
    group reach nothing."""
    g = _gen(4)
    counts, tail, N, K = [70, 3, 0, 65], 30, 144, 264
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w, dy = _ints(g, rows, K), _ints(g, E, N, K), _ints(g, rows, N)
    clean = (sw.swiglu_grouped_mm_fwd(x, w, ends), sw.swiglu_grouped_mm_dgrad(dy, w, ends),
             sw.swiglu_grouped_mm_wgrad(dy, x, ends), sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32),
             sw.swiglu_grouped_fc1_fwd(x, w, ends))
    x, dy = x.clone(), dy.clone()
    x[70:73] = bad  # group 1 alone
    dy[70:73] = bad
    x[sum(counts):] = bad  # rows of no group
    dy[sum(counts):] = bad
    y, dx = sw.swiglu_grouped_mm_fwd(x, w, ends), sw.swiglu_grouped_mm_dgrad(dy, w, ends)
    y1 = sw.swiglu_grouped_fc1_fwd(x, w, ends)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[70:73] = False
    assert _same_bits(y[keep], clean[0][keep]) and _same_bits(dx[keep], clean[1][keep])
    assert _same_bits(y1[keep], clean[4][keep])
    assert float(y[sum(counts):].abs().max()) == 0.0 and float(dx[sum(counts):].abs().max()) == 0.0
    for dw, ref in ((sw.swiglu_grouped_mm_wgrad(dy, x, ends), clean[2]),
                    (sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32), clean[3])):
        assert _same_bits(dw[[0, 2, 3]], ref[[0, 2, 3]])
        assert not bool(torch.isfinite(dw[1]).any())


@pytest.mark.parametrize("N,K", [(136, 72), (2056, 2056)])
def test_long_groups_keep_fp32_precision(sw, N, K):
    """A weight gradient over 13,000 rows of one sign, in fp32.  Each step of 16 rows
    truncates the running sum, by 2^-23 of it at most and half that on average: 256
    steps per segment of 4096 rows stay within 2^-15, where 813 steps in one go
    would be off by 4e-5 on average.  The segments (slices of the sum, where the
    tiles are few) are added with rounding."""
    g = _gen(5)
    rows = 13000
    x, dy = _normal(g, rows, K).abs(), _normal(g, rows, N).abs()
    ends = _ends([rows])
    ref, _ = R.wgrad(dy, x, ends, 1)
    tol = 256 * 2.0 ** -23 + 10 * 2.0 ** -24
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32)
    assert float(((dw.double() - ref).abs() / ref).max()) <= tol
    start = _normal(g, 1, N, K).float()
    more = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=start.clone(), accumulate=True)
    assert float(((more.double() - start.double() - ref).abs() / ref).max()) <= tol


def test_guards_repeats_and_streams(sw):
    """Outputs inside larger buffers: nothing else is written; the same bits each
    time, on another stream, and beside other work."""
    g = _gen(6)
    counts, tail, N, K = [130, 0, 257, 5], 9, 144, 72
    rows, E, ends = sum(counts) + tail, len(counts), _ends(counts)
    x, w, dy = _normal(g, rows, K), _normal(g, E, N, K), _normal(g, rows, N)

    def guarded(shape, dtype):
        n = 1
        for d in shape:
            n *= d
        pat = 0x5a5a if dtype.itemsize == 2 else 0x5a5a5a5a if dtype.itemsize == 4 else 0x5a
        buf = torch.full((n + 512,), pat, device="cuda",
                         dtype={1: torch.uint8, 2: torch.int16, 4: torch.int32}[dtype.itemsize])
        return buf, buf.view(dtype)[256:256 + n].view(shape), pat

    def clean(buf, pat):
        return bool((buf[:256] == pat).all()) and bool((buf[-256:] == pat).all())

    side = torch.cuda.Stream()
    for _ in range(2):
        by, y, py = guarded((rows, N), torch.bfloat16)
        bx, dx, px = guarded((rows, K), torch.bfloat16)
        bw, dw, pw = guarded((E, N, K), torch.float32)
        n = N // 2
        b1, y1, p1 = guarded((rows, n), torch.bfloat16)
        bq, q, pq = guarded((rows, N), torch.float8_e4m3fn)
        bs, s, ps = guarded((rows, 2 * -(-n // 32)), torch.float8_e8m0fnu)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32)
            other_y = sw.swiglu_grouped_mm_fwd(x, w, ends)
        sw.swiglu_grouped_mm_fwd(x, w, ends, y=y)
        sw.swiglu_grouped_mm_dgrad(dy, w, ends, dx=dx)
        sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=dw)
        sw.swiglu_grouped_fc1_fwd(x, w, ends, save="fp8", y=y1, q=q, scales=s)
        torch.cuda.synchronize()
        for buf, pat in ((by, py), (bx, px), (bw, pw), (b1, p1), (bq, pq), (bs, ps)):
            assert clean(buf, pat)
        assert _same_bits(other, dw) and _same_bits(other_y, y)


def test_graph_replays_with_other_groups(sw):
    """The host never reads ends: a captured step follows new groups."""
    g = _gen(7)
    rows, E, N, K = 500, 7, 144, 264
    x, w, dy = _ints(g, rows, K), _ints(g, E, N, K), _ints(g, rows, N)
    ends = _ends([100, 0, 50, 200, 1, 2, 3])

    def step():
        return (sw.swiglu_grouped_mm_fwd(x, w, ends), sw.swiglu_grouped_mm_dgrad(dy, w, ends),
                sw.swiglu_grouped_mm_wgrad(dy, x, ends), sw.swiglu_grouped_fc1_fwd(x, w, ends, save="bf16")[1])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for counts in ([100, 0, 50, 200, 1, 2, 3], [0, 0, 0, 0, 0, 0, 500], [3, 2, 1, 0, 450, 44, 0], [0] * 7):
        ends.copy_(_ends(counts))
        graph.replay()
        torch.cuda.synchronize()
        refs = (R.mm(x, w, ends)[0], R.dgrad(dy, w, ends)[0], R.wgrad(dy, x, ends, E)[0], R.mm(x, w, ends)[0])
        for a, b in zip(out, refs):
            assert _same_bits(a + 0.0, b.bfloat16() + 0.0)


def test_first_call_of_a_thread(sw):
    """A thread that has made no CUDA call yet (as the autograd engine's) gives the
    same bits; also for the dense first product, which encodes its maps likewise."""
    import threading

    g = _gen(10)
    x, w, dy = _normal(g, 70, 72), _normal(g, 2, 128, 72), _normal(g, 70, 128)
    ends = _ends([40, 30])

    def calls():
        return (sw.swiglu_grouped_mm_dgrad(dy, w, ends), sw.swiglu_grouped_mm_wgrad(dy, x, ends),
                sw.swiglu_grouped_fc1_fwd(x, w, ends), sw.swiglu_fc1_fwd(x, w[0]))

    want = calls()
    torch.cuda.synchronize()
    for first in range(4):
        got = []

        def work():
            one = (lambda: sw.swiglu_grouped_mm_dgrad(dy, w, ends), lambda: sw.swiglu_grouped_mm_wgrad(dy, x, ends),
                   lambda: sw.swiglu_grouped_fc1_fwd(x, w, ends), lambda: sw.swiglu_fc1_fwd(x, w[0]))[first]
            got.append(one())
            got.append(calls())
            torch.cuda.synchronize()

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert len(got) == 2 and torch.equal(got[0], want[first])
        assert all(torch.equal(a, b) for a, b in zip(got[1], want))


@pytest.mark.parametrize("counts,n", [([5, 3], 40), ([300, 270, 200, 130], 2056)])
def test_deep_gates(sw, counts, n):
    """Gates from -130 to 130 (integers, so the products are exact): y within one
    bf16 step, subnormal results and zeros included, on both kernels."""
    g = _gen(11)
    rows, E, K = sum(counts), len(counts), 64
    x = torch.zeros(rows, K, device="cuda")
    x[:, 0] = torch.randint(-130, 131, (rows,), generator=g, device="cuda").float()
    x[:, 1] = torch.randint(-8, 9, (rows,), generator=g, device="cuda").float()
    w = torch.zeros(E, 2 * n, K, device="cuda")
    w[:, :n, 0] = 1.0  # the gate is x[0]
    w[:, n:, 1] = torch.randint(-3, 4, (E, n), generator=g, device="cuda").float()
    x, w, ends = x.bfloat16(), w.bfloat16(), _ends(counts)
    p = torch.rand(rows, generator=g, device="cuda")
    ref = R.mm(x, w, ends)[0]
    want = (R.silu64(ref[:, :n]) * ref[:, n:] * p.double()[:, None]).bfloat16()
    y = sw.swiglu_grouped_fc1_fwd(x, w, ends, p)
    assert int((bf16_ordered(y) - bf16_ordered(want)).abs().max()) <= 1


def test_python_layer_refusals(sw):
    g = _gen(12)
    x, w, ends = _ints(g, 20, 16), _ints(g, 2, 32, 16), _ends([12, 8])
    dy = _ints(g, 20, 32)
    for bad in (lambda: sw.swiglu_grouped_mm_fwd(x.float(), w, ends), lambda: sw.swiglu_grouped_mm_fwd(x, w.float(), ends),
                lambda: sw.swiglu_grouped_mm_fwd(x, w, ends.long()), lambda: sw.swiglu_grouped_mm_fwd(x, w, ends[:1]),
                lambda: sw.swiglu_grouped_mm_fwd(x, w, ends.cpu()), lambda: sw.swiglu_grouped_mm_fwd(x.cpu(), w, ends),
                lambda: sw.swiglu_grouped_mm_fwd(dy, w, ends), lambda: sw.swiglu_grouped_mm_fwd(x[:, ::2], w, ends),
                lambda: sw.swiglu_grouped_mm_fwd(x, w.transpose(1, 2), ends), lambda: sw.swiglu_grouped_mm_fwd(x, w[0], ends),
                lambda: sw.swiglu_grouped_mm_fwd(x, w, ends, y=dy[:, :16]), lambda: sw.swiglu_grouped_mm_dgrad(x, w, ends),
                lambda: sw.swiglu_grouped_mm_wgrad(dy, x[:10], ends), lambda: sw.swiglu_grouped_mm_wgrad(dy, x, ends, accumulate=True),
                lambda: sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float16),
                lambda: sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=w, accumulate=True),
                lambda: sw.swiglu_grouped_fc1_fwd(x, w[:, :31], ends), lambda: sw.swiglu_grouped_fc1_fwd(x, w, ends, x[:, 0]),
                lambda: sw.swiglu_grouped_fc1_fwd(x, w, ends, torch.rand(19, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sw.SwigluError, match="SHAPE"):  # widths that are no multiple of 8
        sw.swiglu_grouped_mm_fwd(_ints(g, 4, 12), _ints(g, 1, 8, 12), _ends([4]))
    square = _ints(g, 20, 32)
    with pytest.raises(sw.SwigluError, match="ALIAS"):
        sw.swiglu_grouped_mm_fwd(square, _ints(g, 2, 32, 32), ends, y=square)


@pytest.mark.parametrize("N,K", [(264, 520), (72, 64), (1032, 1288)])
def test_weight_gradient_of_every_remainder(sw, N, K):
    """Groups of 0 to 130 rows, in both orders: every number of rows in a group's last
    block, next to a group of NaN, and at the end of the tensor."""
    for counts in (list(range(131)), list(range(130, -1, -1))):
        bad = counts.index(61)
        rows, g = sum(counts), _gen(N + counts[0])
        x, dy = _ints(g, rows, K), _ints(g, rows, N)
        first = sum(counts[:bad])
        x[first:first + 61], dy[first:first + 61] = math.nan, math.nan
        for dtype in (torch.bfloat16, torch.float32):
            dw = sw.swiglu_grouped_mm_wgrad(dy, x, _ends(counts), dtype=dtype)
            r0 = 0
            for e, c in enumerate(counts):
                ref = (dy[r0:r0 + c].double().T @ x[r0:r0 + c].double()).to(dtype)
                r0 += c
                if e == bad:
                    assert bool(dw[e].isnan().all())
                else:
                    assert torch.equal(dw[e], ref), f"group of {c} rows, {dtype}"
    assert sw.grouped_timeout_flag() == 0


def test_many_groups(sw):
    """1024 groups (the most of one call), most of them empty."""
    g = _gen(8)
    E, N, K = 1024, 64, 64
    counts = torch.zeros(E, dtype=torch.int64)
    counts[torch.arange(0, E, 37)] = torch.arange(0, E, 37) % 50
    ends = _ends(counts.tolist())
    rows = int(counts.sum()) + 5
    x, w, dy = _ints(g, rows, K), _ints(g, E, N, K), _ints(g, rows, N)
    assert _same_bits(sw.swiglu_grouped_mm_fwd(x, w, ends) + 0.0, R.mm(x, w, ends)[0].bfloat16() + 0.0)
    assert _same_bits(sw.swiglu_grouped_mm_wgrad(dy, x, ends) + 0.0, R.wgrad(dy, x, ends, E)[0].bfloat16() + 0.0)


def test_empty(sw):
    w = torch.randn(3, 16, 8, device="cuda").bfloat16()
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 8, device="cuda").bfloat16(), torch.empty(0, 16, device="cuda").bfloat16()
    assert sw.swiglu_grouped_mm_fwd(x, w, ends).shape == (0, 16)
    assert sw.swiglu_grouped_mm_dgrad(dy, w, ends).shape == (0, 8)
    assert sw.swiglu_grouped_fc1_fwd(x, w, ends, save="fp8")[1].shape == (0, 16)
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=torch.ones(3, 16, 8, device="cuda"))
    assert float(dw.abs().max()) == 0.0
    kept = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=torch.ones(3, 16, 8, device="cuda"), accumulate=True)
    assert float(kept.min()) == 1.0


def test_large_offsets(sw):
    """Element offsets past 2^31 in x, W, y and dW: sampled rows and experts."""
    g = _gen(9)
    E, N, K = 130, 4096, 4104  # W: 2.2e9 elements
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    for e in range(0, E, 10):
        w[e:e + 10] = _ints(g, 10, N, K, top=1)
    counts = [0] * E
    counts[0], counts[127], counts[129] = 5, 40, 33
    ends = _ends(counts)
    x = _ints(g, 78, K, top=1)
    assert _same_bits(sw.swiglu_grouped_mm_fwd(x, w, ends) + 0.0, R.mm(x, w, ends)[0].bfloat16() + 0.0)
    dy = _ints(g, 78, N, top=1)
    assert _same_bits(sw.swiglu_grouped_mm_dgrad(dy, w, ends) + 0.0, R.dgrad(dy, w, ends)[0].bfloat16() + 0.0)
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends)
    for e, (a, b) in ((0, (0, 5)), (1, (5, 5)), (127, (5, 45)), (128, (45, 45)), (129, (45, 78))):
        ref = dy[a:b].double().T @ x[a:b].double()
        assert _same_bits(dw[e] + 0.0, ref.bfloat16() + 0.0)
    del w, dw
    rows, N, K = 300001, 64, 8192  # x: 2.46e9 elements
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, 30000):
        x[at:at + 30000] = _ints(g, x[at:at + 30000].shape[0], K, top=1)
    w = _ints(g, 2, N, K, top=1)
    ends = _ends([270000, 30000])
    y = sw.swiglu_grouped_mm_fwd(x, w, ends)
    dx = sw.swiglu_grouped_mm_dgrad(y, w, ends)
    pick = torch.tensor([0, 262143, 262144, 269999, 270000, 299999, 300000], device="cuda")
    which = torch.tensor([0, 0, 0, 0, 1, 1, 1], device="cuda")
    live = torch.tensor([1, 1, 1, 1, 1, 1, 0], device="cuda").double()[:, None]
    ref = torch.einsum("rk,rnk->rn", x[pick].double(), w[which].double()) * live
    assert _same_bits(y[pick] + 0.0, ref.bfloat16() + 0.0)
    ref = torch.einsum("rn,rnk->rk", y[pick].double(), w[which].double()) * live
    assert _same_bits(dx[pick] + 0.0, ref.bfloat16() + 0.0)


@pytest.mark.parametrize("N,K,scale", [(136, 72, 1), (1032, 1288, 8)])
@pytest.mark.parametrize("some", [True, False])
def test_accumulating_leaves_empty_groups_as_they_are(sw, N, K, scale, some):
    """dW of a group without rows keeps its bits: -0, subnormals, infinities and NaNs
    with a payload among them; next to it the sum is added, subnormals kept.  The
    wider product is the CTA pairs', the other one is split."""
    g = _gen(13)
    counts = [0, 40 * scale, 0, 9 * scale, 0] if some else [0] * 5
    rows, E, ends = sum(counts) + 7, 5, _ends(counts)
    x, dy = _ints(g, rows, K), torch.zeros(rows, N, device="cuda").bfloat16()
    dy[:, ::3] = _ints(g, rows, N)[:, ::3]
    odd = torch.tensor([-2 ** 31, 1, 0x7fffff, 0x7fc01234, 0x7f800000, 0x3f800000, 5 - 2 ** 31, -0x345678],
                       dtype=torch.int32, device="cuda")
    start = odd.repeat(E * N * K // 8).view(E, N, K)
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=start.clone().view(torch.float32), accumulate=True)
    ref, _ = R.wgrad(dy, x, ends, E)
    want = start.view(torch.float32) + ref.float()
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e].view(torch.int32), start[e])
        else:  # (the sums are integers, exact; a NaN need not keep its payload)
            same = (dw[e] == want[e]) | (dw[e].isnan() & want[e].isnan())
            assert bool(same.all())
