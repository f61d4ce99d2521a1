"""The 4-bit products of many rows, several tiles to each pair of CTAs: the stages' ring and
the scales' slots wrap, both accumulators and the columns they share are in use, tiles are
taken from the pairs that have not started.

By the rule that chooses, the kernel for few rows would cost 1.4 to 6 times as much at each of
these sizes: they are the pairs', with 140 to 730 tiles for 76 of them.  Codes and scales are such
that every sum fits the 24 bits of fp32 in any order, so products are held to equality."""
import pytest
import torch

import mx4_reference as R
from test_mx4_gpu import check_mlp, gen, inputs, mlp_case, random_codes, sw  # noqa: F401 (sw: fixture)

pytestmark = pytest.mark.gpu
BF16, E8M0 = torch.bfloat16, torch.float8_e8m0fnu


def operand(g, rows, nb, low, high, parts=1):
    """(values in 64 bits, q, scales) of random codes."""
    code, c = random_codes(g, rows, nb, low, high)
    q, scales = R.pack(code, c, parts)
    return R.values(code, c), q, scales.view(E8M0)


# rows and columns that end anywhere in a tile; 1, 2, 8 and 13 stages, the last one whole or not
PRODUCTS = [(8192, 5504, 2), (8193, 5504, 9), (8224, 5503, 2), (8352, 5503, 2), (8352, 5496, 8), (8352, 5504, 64),
            (8193, 5503, 64), (4128, 5505, 100), (4127, 5520, 97), (160, 60000, 2), (160, 60001, 2), (160, 59992, 9),
            (60001, 160, 2), (20000, 1000, 33)]


@pytest.mark.parametrize("M,N,nb", PRODUCTS)
def test_mm_exact(sw, M, N, nb):
    """Whole packs, 16-byte pieces and rows of any length, each several times over."""
    g = gen(M + N + nb)
    a, *x = operand(g, M, nb, 126, 129)
    b, *w = operand(g, N, nb, 125, 128)
    want = a @ b.T
    # units of 1/4 * 2^-3; 12 and 6 are the largest values
    assert 32 * nb * 12 * 6 < 2 ** 24 * 2.0 ** -5
    want = want.to(BF16)
    buf = torch.full((M * N + 32,), 7.0, dtype=BF16, device="cuda")
    for start in (0, 0, 0, 16, 8, 3):
        y = buf[start:start + M * N].view(M, N)
        y.fill_(5.0)
        sw.swiglu_mx4_mm_fwd(*x, *w, y=y)
        assert torch.equal(y, want)
        assert bool((buf[start + M * N:] == 7).all()) and bool((buf[:start] == 7).all())
        buf.fill_(7.0)
    assert sw.mx4_timeout_flag() == 0


@pytest.mark.parametrize("M,N,K", [(8352, 5503, 64), (8352, 5504, 320), (4100, 5504, 2080)])
def test_mm_keeps_nan_to_its_row_and_column(sw, M, N, K):
    g = gen(M)
    a, xq, xs = operand(g, M, K // 32, 126, 128)
    b, wq, ws = operand(g, N, K // 32, 126, 128)
    for q, scales, rows, bad in ((xq, xs, M, (1, 300, M - 1)), (wq, ws, N, (0, 255, N - 2))):
        s = scales.view(torch.uint8)
        for r in bad:  # the last block of the row is NaN
            blk = K // 32 - 1
            s[r // 128, blk // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + blk % 4] = 255
            q[r, 16 * blk:] = 0
    y = sw.swiglu_mx4_mm_fwd(xq, xs, wq, ws)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[[1, 300, M - 1]], nan[:, [0, 255, N - 2]] = True, True
    assert torch.equal(torch.isnan(y), nan)
    want = (a @ b.T).to(BF16)
    assert torch.equal(y[~nan], want[~nan])


@pytest.mark.parametrize("M,H,n", [(20000, 64, 1000), (20001, 256, 1000), (19744, 288, 1031), (9000, 2048, 1024),
                                   (5000, 3200, 2000), (5153, 96, 4097), (2500, 160, 8200)])
def test_gated_product_as_of_few_rows(sw, M, H, n):
    """The activation's codes: W2 is the identity, so the result is the rounded activation
    itself, equal to that of 64 rows at a time, which the kernel for few rows computes (the
    sums are exact in both; from them on both do the same operations)."""
    g = gen(M + H + n)
    nb = -(-H // 32)
    assert 32 * nb * 12 * 6 < 2 ** 24 * 2.0 ** -5
    x = operand(g, M, nb, 126, 129)[0].to(BF16)
    w1 = operand(g, 2 * n, nb, 122, 125, 2)[1:]
    w2 = sw.swiglu_mx4_quantize(torch.eye(n, device="cuda"))
    out = sw.swiglu_mx4_mlp_fwd(x, *w1, *w2)
    want = torch.cat([sw.swiglu_mx4_mlp_fwd(x[r:r + 64], *w1, *w2) for r in range(0, M, 64)])
    assert torch.equal(out, want)
    assert float((out != 0).float().mean()) > 0.2  # not of nothing
    for _ in range(3):
        assert torch.equal(out, sw.swiglu_mx4_mlp_fwd(x, *w1, *w2))
    assert sw.mx4_timeout_flag() == 0


@pytest.mark.parametrize("M,H,n,N", [(2304, 4096, 3000, 4096), (2500, 256, 8200, 264), (4128, 200, 2500, 2001)])
def test_mlp(sw, M, H, n, N):
    x, w1, w2 = mlp_case(M, H, n, N, seed=M)
    a, b = sw.swiglu_mx4_quantize(w1, 2), sw.swiglu_mx4_quantize(w2)
    out = sw.swiglu_mx4_mlp_fwd(x, *a, *b)
    check_mlp(out, x, w1, w2)
    for _ in range(3):
        assert torch.equal(out, sw.swiglu_mx4_mlp_fwd(x, *a, *b))
    x[M - 70, 3] = float("nan")
    bad = sw.swiglu_mx4_mlp_fwd(x, *a, *b)
    keep = torch.arange(M, device="cuda") != M - 70
    assert bool(torch.isnan(bad[M - 70]).all()) and torch.equal(bad[keep], out[keep])
    assert sw.mx4_timeout_flag() == 0


@pytest.mark.parametrize("M,N,K", [(3000, 4000, 3500), (8352, 5503, 2000)])
def test_mm(sw, M, N, K):
    """Values of every size, against 64 bits within the sums' bound."""
    from test_mx4_gpu import check_product

    x, w = inputs(M, K, BF16, 1), inputs(N, K, BF16, 2)
    a, b = sw.swiglu_mx4_quantize(x), sw.swiglu_mx4_quantize(w)
    y = sw.swiglu_mx4_mm_fwd(*a, *b)
    check_product(y, R.rounded(x), R.rounded(w), K)
    for _ in range(3):
        assert torch.equal(y, sw.swiglu_mx4_mm_fwd(*a, *b))
