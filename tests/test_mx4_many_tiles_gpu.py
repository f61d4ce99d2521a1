"""The 4-bit products of many rows, several tiles to each pair of CTAs: the stages' ring and
the scales' slots wrap, both accumulators and the columns they share are in use, tiles are
taken from the pairs that have not started.

By the rule that chooses, the kernel for few rows would cost 1.4 to 6 times as much at each of
these sizes: they are the pairs', with 140 to 730 tiles for 76 of them.  Codes and scales are such
that every sum fits the 24 bits of fp32 in any order, so products are held to equality."""
import pytest
import torch

import mx4_reference as R
from test_mx4_gpu import gen, random_codes, sw  # noqa: F401 (sw: fixture)

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
