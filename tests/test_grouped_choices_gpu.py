"""The grouped products in every way that they are computed: by pairs of CTAs, and with
the contraction in 1, 2, 4 and 8 slices.  Each size below is checked to take the way that
it stands for (test_grouped_choices.py does so without a GPU as well), so that another
choice between them cannot take a kernel out of the tests unnoticed.

Inputs are small integers: every product and partial sum is exact, so the results equal
the exact ones rounded once, bit for bit (y of the first product: one bf16 step, it
passes through the exponential)."""
import pytest
import torch

import moe_reference as R
from grouped_choices import CASES, counts_of
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


def _ends(counts):
    return torch.tensor(counts, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


def _bits(t):
    return (t + 0.0).view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.dtype.itemsize])  # (one zero)


class Guarded:
    """A tensor inside a larger buffer of a pattern."""

    def __init__(self, shape, dtype):
        n = torch.Size(shape).numel()
        self.raw = torch.full((n * dtype.itemsize + 1024,), 0x5a, dtype=torch.uint8, device="cuda")
        self.t = self.raw[512:512 + n * dtype.itemsize].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:512] == 0x5a).all()) and bool((self.raw[-512:] == 0x5a).all())


class Problem:
    """Inputs of one product and its call; ``exact(ends)`` the 64-bit result."""

    def __init__(self, sw, case):
        product, dtype, slices, rows, E, N, K = case
        assert sw.grouped_slices(product, rows, E, N, K, dtype) == slices
        g = torch.Generator(device="cuda").manual_seed(rows + 3 * N + 7 * K)
        self.sw, self.product, self.dtype, self.E = sw, product, dtype, E
        self.counts, self.tail = counts_of(rows, E)
        self.rows, self.n = rows, N
        n_rows = 2 * N if product == "fc1" else N
        fc1 = product == "fc1"
        self.x = _ints(g, rows, K, top=1 if fc1 else 3)
        self.w = _ints(g, E, n_rows, K, top=2 if fc1 else 3)
        self.dy = _ints(g, rows, n_rows)
        self.start = _ints(g, E, N, K).float() if dtype == torch.float32 else None
        shape = {"fc1": (rows, N), "mm": (rows, N), "dgrad": (rows, K), "wgrad": (E, N, K)}[product]
        self.out = Guarded(shape, dtype)
        if fc1:
            self.fc1 = Guarded((rows, 2 * N), torch.bfloat16)
            self.q = Guarded((rows, 2 * N), torch.float8_e4m3fn)
            self.scales = Guarded((rows, 2 * -(-N // 32)), torch.float8_e8m0fnu)
        self.probs = torch.rand(rows, generator=g, device="cuda") if fc1 else None

    def run(self, ends):
        sw = self.sw
        if self.product == "mm":
            sw.swiglu_grouped_mm_fwd(self.x, self.w, ends, y=self.out.t)
        elif self.product == "dgrad":
            sw.swiglu_grouped_mm_dgrad(self.dy, self.w, ends, dx=self.out.t)
        elif self.product == "wgrad":
            if self.start is not None:
                self.out.t.copy_(self.start)
            sw.swiglu_grouped_mm_wgrad(self.dy, self.x, ends, dw=self.out.t, accumulate=self.start is not None)
        else:
            sw.swiglu_grouped_fc1_fwd(self.x, self.w, ends, self.probs, y=self.out.t, save="bf16", fc1=self.fc1.t)
            y = self.out.t.clone()
            sw.swiglu_grouped_fc1_fwd(self.x, self.w, ends, self.probs, y=self.out.t, save="fp8", q=self.q.t,
                                      scales=self.scales.t)
            assert torch.equal(_bits(y), _bits(self.out.t)) or bool(y.isnan().any())

    def check(self, ends, keep):
        """Against the exact result, in the rows (weight gradient: groups) `keep`."""
        if self.product == "wgrad":
            want = R.wgrad(self.dy, self.x, ends, self.E)[0]
            want = (want if self.start is None else want + self.start.double()).to(self.dtype)
        elif self.product == "dgrad":
            want = R.dgrad(self.dy, self.w, ends)[0].bfloat16()
        else:
            want = R.mm(self.x, self.w, ends)[0]
        got = self.out.t
        if self.product != "fc1":
            assert torch.equal(_bits(got[keep]), _bits(want.to(self.dtype)[keep]))
        else:
            n = self.n
            y = (R.silu64(want[:, :n]) * want[:, n:] * self.probs.double()[:, None]).bfloat16()
            assert int((bf16_ordered(got[keep]) - bf16_ordered(y[keep])).abs().max()) <= 1
            assert torch.equal(_bits(self.fc1.t[keep]), _bits(want.bfloat16()[keep]))
            q, codes = R.checkpoint(want[keep])
            assert torch.equal(self.scales.t[keep].view(torch.uint8).long(), codes)
            assert torch.equal(self.q.t[keep].float().double(), q)
        outs = [self.out] + ([self.fc1, self.q, self.scales] if self.product == "fc1" else [])
        assert all(o.intact() for o in outs), "written outside of the result"


def _name(case):
    product, dtype, slices, rows, E, N, K = case
    return f"{product}{'32' if dtype == torch.float32 else ''}-{slices or 'pairs'}-{rows}x{E}x{N}x{K}"


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_exact_next_to_nan(sw, case):
    """One group and the rows of no group are NaN: nothing else takes it in, every value
    is exact, and nothing is written outside of the results."""
    p = Problem(sw, case)
    ends, live = _ends(p.counts), sum(p.counts)
    a, b = sum(p.counts[:2]), sum(p.counts[:3])
    if p.product == "wgrad":
        keep = torch.arange(p.E, device="cuda") != 2
    else:
        keep = torch.ones(p.rows, dtype=torch.bool, device="cuda")
        keep[a:b] = False
    clean = [t.clone() for t in (p.x, p.dy)]
    for t in (p.x, p.dy):
        t[a:b] = float("nan")
        t[live:] = float("nan")
    p.run(ends)
    if p.product == "wgrad":
        assert bool(p.out.t[2].isnan().all())
    else:
        assert bool(p.out.t[a:b].isnan().all())
        assert not bool(p.out.t[live:].any())
    p.x, p.dy = clean
    p.check(ends, keep)


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_other_groups_in_a_replay(sw, case):
    """The host never reads ends: a captured call follows new ones, whatever they hold."""
    p = Problem(sw, case)
    ends = _ends(p.counts)
    p.run(ends)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _captured(p, ends)
    rows, E = p.rows, p.E
    whole = slice(None)
    for values in ([rows // 2] * E, [rows + 5] + [-3] * (E - 1), [0] * (E - 1) + [rows],
                   [(e * 977) % (rows + 9) - 4 for e in range(E)], [-2 ** 31] * E, [2 ** 31 - 1] * E):
        ends.copy_(torch.tensor(values, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        p.check(ends, whole)


def _captured(p, ends):
    """The call without the comparison of run()."""
    sw = p.sw
    if p.product == "fc1":
        sw.swiglu_grouped_fc1_fwd(p.x, p.w, ends, p.probs, y=p.out.t, save="bf16", fc1=p.fc1.t)
        sw.swiglu_grouped_fc1_fwd(p.x, p.w, ends, p.probs, y=p.out.t, save="fp8", q=p.q.t, scales=p.scales.t)
    else:
        p.run(ends)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "fc1"], ids=_name)
def test_deep_gates(sw, case):
    """Gates from -130 to 130: y within one bf16 step, subnormal results and zeros included."""
    p = Problem(sw, case)
    g = torch.Generator(device="cuda").manual_seed(1)
    p.x.zero_(), p.w.zero_()
    p.x[:, 0] = torch.randint(-130, 131, (p.rows,), generator=g, device="cuda").bfloat16()
    p.x[:, 1] = _ints(g, p.rows, top=8)
    p.w[:, :p.n, 0] = 1.0  # the gate is x[0]
    p.w[:, p.n:, 1] = _ints(g, p.E, p.n)
    ends = _ends(p.counts)
    p.run(ends)
    p.check(ends, slice(None))


def test_many_groups_by_pairs(sw):
    """1024 groups (the most of one call), most of them empty, by pairs of CTAs."""
    g = torch.Generator(device="cuda").manual_seed(8)
    E, N, K = 1024, 264, 136
    counts = torch.zeros(E, dtype=torch.int64)
    counts[torch.arange(0, E, 7)] = torch.arange(0, E, 7) % 300
    rows, ends = int(counts.sum()) + 5, _ends(counts.tolist())
    x, dy, w = _ints(g, rows, K), _ints(g, rows, N), _ints(g, E, N, K)
    assert sw.grouped_slices("wgrad", rows, E, N, K) == 0 and sw.grouped_slices("mm", rows, E, N, K) == 0
    assert torch.equal(_bits(sw.swiglu_grouped_mm_wgrad(dy, x, ends)), _bits(R.wgrad(dy, x, ends, E)[0].bfloat16()))
    assert torch.equal(_bits(sw.swiglu_grouped_mm_fwd(x, w, ends)), _bits(R.mm(x, w, ends)[0].bfloat16()))


@pytest.mark.parametrize("checkpoint", ["fp8", "bf16"])
def test_module_by_pairs(sw, checkpoint):
    """The layer at sizes where its six products go by pairs; tolerances as for its other
    tests (bf16 roundings: 1e-2 in the Frobenius norm)."""
    from gate_up_swiglu_gb300.experts import ExpertsSwiGLU, group_ends

    g = torch.Generator(device="cuda").manual_seed(2)
    counts, H, n = [700, 0, 33, 1, 750], 1288, 1288
    rows, E = sum(counts) + 16, 5
    for product, N, K in (("fc1", n, H), ("mm", H, n), ("dgrad", H, n), ("dgrad", 2 * n, H), ("wgrad", H, n),
                          ("wgrad", 2 * n, H)):
        assert sw.grouped_slices(product, rows, E, N, K) == 0
    x = torch.randn(rows, H, generator=g, device="cuda").bfloat16().requires_grad_(True)
    probs = torch.rand(rows, generator=g, device="cuda").requires_grad_(True)
    dout = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    c = torch.tensor(counts, device="cuda")
    m = ExpertsSwiGLU(E, H, n, checkpoint=checkpoint, device="cuda")
    out = m(x, c, probs)
    out.backward(dout)
    ends, w1, w2, xd, pd = group_ends(c), m.w1.detach(), m.w2.detach(), x.detach(), probs.detach()
    f = R.mm(xd, w1, ends)[0]
    y = R.silu64(f[:, :n]) * f[:, n:] * pd.double()[:, None]
    kept = f
    if checkpoint == "fp8":
        kept = R.restored(*sw.swiglu_grouped_fc1_fwd(xd, w1, ends, pd, save="fp8")[1:])
    dfc1, dp, y2, _ = R.swiglu_bwd(R.dgrad(dout, w2, ends)[0], kept, pd)
    for name, got, want in (("out", out, R.mm(y, w2, ends)[0]), ("dx", x.grad, R.dgrad(dfc1, w1, ends)[0]),
                            ("dprobs", probs.grad, dp), ("dw1", m.w1.grad, R.wgrad(dfc1, xd, ends, E)[0]),
                            ("dw2", m.w2.grad, R.wgrad(dout, y2, ends, E)[0])):
        assert float((got.detach().double() - want).norm() / want.norm()) < 1e-2, name


def test_bf16_weight_gradients_over_many_rows(sw):
    """A bf16 dW over more rows than one running sum may have, by pairs: long and short
    groups in turn, with NaN rows behind; integers, so that every sum is exact."""
    g = torch.Generator(device="cuda").manual_seed(3)
    counts, N, K = [300, 270_000, 0, 5, 131_072, 140_001, 700], 1032, 1288
    rows, E, ends = sum(counts) + 100, len(counts), _ends(counts)
    assert sw.grouped_slices("wgrad", rows, E, N, K) == 0
    x, dy = _ints(g, rows, K, top=1), _ints(g, rows, N, top=2)
    x[-100:], dy[-100:] = float("nan"), float("nan")
    got = sw.swiglu_grouped_mm_wgrad(dy, x, ends)
    at = 0
    for e, c in enumerate(counts):
        want = torch.zeros(N, K, dtype=torch.float64, device="cuda")
        for r in range(at, at + c, 65536):
            t = min(r + 65536, at + c)
            want += dy[r:t].double().T @ x[r:t].double()
        at += c
        assert torch.equal(_bits(got[e]), _bits(want.bfloat16())), f"group of {c} rows"


@pytest.mark.parametrize("rows,N,K,slices", [(600_000, 2056, 2048, 0), (600_000, 128, 136, 8), (1_200_000, 72, 72, 8)])
def test_bf16_weight_gradients_keep_their_precision(sw, rows, N, K, slices):
    """Many rows of one sign.  Each step of 16 rows truncates the running sum by less
    than 2^-23 of it, so 131,072 rows lose at most 2^13 2^-23 = 2^-10; with the rounding
    to bf16 (8 significant bits: 2^-8) and of the additions every value is within 2^-8 +
    2^-10 + 2^-20.  One running sum of 600,000 would lose 3.8e-3 on average."""
    g = torch.Generator(device="cuda").manual_seed(4)
    assert sw.grouped_slices("wgrad", rows, 1, N, K) == slices
    x = torch.randn(rows, K, generator=g, device="cuda").bfloat16().abs()
    dy = torch.randn(rows, N, generator=g, device="cuda").bfloat16().abs()
    some = torch.arange(0, N, 37, device="cuda")  # rows of dW
    got = sw.swiglu_grouped_mm_wgrad(dy, x, _ends([rows]))[0][some]
    want = torch.zeros(len(some), K, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 65536):
        want += dy[r:r + 65536, some].double().T @ x[r:r + 65536].double()
    assert float(((got.double() - want).abs() / want).max()) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -20


@pytest.mark.parametrize("counts,N,K,slices", [([13_000, 0, 300, 4000], 1288, 1544, 0), ([5200, 40], 1032, 264, 4),
                                               ([13_000], 136, 72, 8)])
def test_fp32_weight_gradients_keep_their_precision(sw, counts, N, K, slices):
    """Rows of one sign, in fp32.  A sum of 512 rows takes 32 steps, each of which truncates
    it by less than 2^-23 of it; the sums are added with rounded additions, one per 512
    rows (and per slice, and one to what dW holds)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, E, ends = sum(counts) + 9, len(counts), _ends(counts)
    assert sw.grouped_slices("wgrad", rows, E, N, K, torch.float32) == slices
    x = torch.randn(rows, K, generator=g, device="cuda").bfloat16().abs()
    dy = torch.randn(rows, N, generator=g, device="cuda").bfloat16().abs()
    want = R.wgrad(dy, x, ends, E)[0]
    tol = 32 * 2.0 ** -23 + (-(-max(counts) // 512) + 9) * 2.0 ** -24
    dw = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dtype=torch.float32)
    assert bool(((dw.double() - want).abs() <= tol * want).all())
    start = torch.randn(E, N, K, generator=g, device="cuda").abs()
    more = sw.swiglu_grouped_mm_wgrad(dy, x, ends, dw=start.clone(), accumulate=True)
    assert bool(((more.double() - start.double() - want).abs() <= tol * (want + start.double())).all())
