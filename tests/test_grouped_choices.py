"""The choice between the kernels of the grouped products, which the host makes from the
sizes alone (no GPU)."""
import pytest
import torch

from grouped_choices import CASES, counts_of


@pytest.fixture(scope="module")
def sw():
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


@pytest.mark.parametrize("case", CASES)
def test_sizes_take_the_way_they_stand_for(sw, case):
    product, dtype, slices, rows, E, N, K = case
    assert sw.grouped_slices(product, rows, E, N, K, dtype) == slices
    counts, tail = counts_of(rows, E)
    assert sum(counts) + tail == rows and min(counts) == counts[1] == 0 and counts[2] > 0 and counts[0] > 0


def test_every_way_has_a_size():
    for product in ("fc1", "mm", "dgrad", "wgrad"):
        for dtype in (torch.bfloat16,) + ((torch.float32,) if product == "wgrad" else ()):
            assert {c[2] for c in CASES if c[:2] == (product, dtype)} == {0, 1, 2, 4, 8}


def test_refusals(sw):
    assert sw.grouped_slices("mm", 0, 2, 16, 16) == 0
    for bad in (dict(product="fc2"), dict(dtype=torch.float16)):
        kw = dict(product="mm", rows=4, groups=2, N=16, K=16)
        with pytest.raises(ValueError):
            sw.grouped_slices(**{**kw, **bad})
    for bad in (dict(rows=-1), dict(groups=0), dict(groups=1025), dict(N=12), dict(K=0), dict(N=1 << 29, product="fc1")):
        kw = dict(product="mm", rows=4, groups=2, N=16, K=16)
        with pytest.raises(sw.SwigluError, match="SHAPE"):
            sw.grouped_slices(**{**kw, **bad})
    assert sw.lib.swiglu_grouped_slices(1, 4, 2, 16, 16, 1, None) == -1
