"""The workloads of the MLP sublayer's operators: their calls of the package are calls it
takes, and compute what the plain forms compute."""
import importlib.util
import os
import random
import sys
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("op,call,tensors", [("mm", "swiglu_mx4_mm_fwd", 4), ("mlp", "swiglu_mx4_mlp_fwd", 5)])
def test_codes_reach_the_package_as_bytes(cases, monkeypatch, op, call, tensors):
    """Whatever type prepare() keeps them in (no GPU: a stand-in takes the call)."""
    seen = []
    package = types.ModuleType("gate_up_swiglu_gb300")
    setattr(package, call, lambda *a: seen.append(a))
    monkeypatch.setitem(sys.modules, "gate_up_swiglu_gb300", package)
    monkeypatch.setattr(cases, "own", True)
    g = torch.Generator().manual_seed(0)
    part = lambda rows, n, parts=1: cases._quantize(torch.randn(rows, n, generator=g), parts)  # noqa: E731
    x, w1, w2 = torch.randn(3, 64, generator=g).bfloat16(), part(80, 64, 2), part(64, 40)
    state = {"case": {"op": op}, "x": part(3, 64) if op == "mm" else x, "w": part(16, 64), "w1": w1, "w2": w2}
    cases.run(state)
    (args,) = seen
    assert len(args) == tensors
    pairs = args if op == "mm" else args[1:]
    given = (*state["x"], *state["w"]) if op == "mm" else (*w1, *w2)
    for k, (t, s) in enumerate(zip(pairs, given)):
        assert t.dtype is (torch.uint8, torch.float8_e8m0fnu)[k % 2] and t.is_contiguous()
        assert torch.equal(t.view(torch.uint8).long(), (s.view(torch.uint8) if k % 2 else s).long())


SMALL = [dict(op="norm_fwd", rows=9, n=100, dtype="bf16", w=True, b=True, pad=3),
         dict(op="norm_fwd", rows=40, n=257, dtype="f32", w=False, b=False, pad=0),
         dict(op="norm_bwd", rows=33, n=512, dtype="bf16", w=True, b=True, pad=0),
         dict(op="norm_bwd", rows=17, n=111, dtype="f32", w=True, b=False, pad=16),
         dict(op="quantize", rows=130, n=300, dtype="bf16", pad=0), dict(op="quantize", rows=7, n=95, dtype="f32", pad=1),
         dict(op="mm", rows=5, N=130, K=96), dict(op="mm", rows=300, N=257, K=1000),
         dict(op="mlp", rows=3, H=200, n=100), dict(op="mlp", rows=129, H=256, n=300)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SMALL, ids=lambda c: f"{c['op']}-{c['rows']}")
def test_package_and_plain_form(cases, monkeypatch, case):
    """Both against the definition in 64 bits, in the norm of the whole result.  16-bit results:
    half a step an element, and as much for the sums.  fp32 results: a sum is within 64 units
    of 2^-24 of that of its absolute values, and no result hangs on more than two that are
    larger than itself by up to two: 2^-16.  MLP: activations near a code's border fall on
    either side, a step of 2^-2 of few of them: 2^-7 in all."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from conftest import build_library

    build_library()
    state, want = cases.prepare(case, 3), cases.exact(case, 3)

    def leaves(v):
        return list(v.values()) if isinstance(v, dict) else list(v) if isinstance(v, (list, tuple)) else [v]

    for own in (False, True):
        monkeypatch.setattr(cases, "own", own)
        got = cases.run(state)
        assert len(leaves(got)) == len(leaves(want))
        for a, b in zip(leaves(got), leaves(want)):
            assert (a is None) == (b is None)
            if a is None:
                continue
            assert a.shape == b.shape
            bound = 2.0 ** -16 if a.dtype is torch.float32 else 2.0 ** -7  # bf16: eps = 2^-7
            assert float((a.double() - b).norm()) <= bound * float(b.norm()) + 1e-30


def test_drawn_cases_stay_in_their_ranges(cases):
    rng = random.Random(0)
    for _ in range(300):
        c = cases.draw(rng)
        w = cases.work(c)
        assert c["rows"] >= 1 and w["bytes"] > 0 and w["flops"] > 0
        assert w["flops"] <= 6 * 8192 * 4096 * 14336
