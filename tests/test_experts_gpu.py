"""The experts' MLP (grouped products + activation + checkpoint) end to end.

Tolerances: bf16 products and bf16 intermediate results give relative Frobenius
errors around 2^-9 per rounding; 1e-2 as for the fc1 module.  With the 8-bit
checkpoint the gradients are compared, to the same 1e-2, with the 64-bit ones at
the values that the checkpoint stands for, and with those of the exact fc1 to
0.1: a code is within 2^-4 of its value, 2^-5.3 in the mean square, and two or
three such factors meet in each term."""
import pytest
import torch

import moe_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from conftest import build_library

    build_library()
    import gate_up_swiglu_gb300 as sw

    return sw


def _inputs(counts, tail, H, n, seed, probs=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, E = sum(counts) + tail, len(counts)
    x = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    w1 = (torch.randn(E, 2 * n, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    w2 = (torch.randn(E, H, n, generator=g, device="cuda") * n ** -0.5).bfloat16()
    p = torch.rand(rows, generator=g, device="cuda") if probs else None
    dout = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    return x, w1, w2, p, dout, torch.tensor(counts, device="cuda")


def _reference(x, w1, w2, p, dout, ends, fc1=None):
    """64-bit out and gradients; fc1: the values the backward works on."""
    f = R.mm(x, w1, ends)[0]
    n = f.shape[1] // 2
    y = R.silu64(f[:, :n]) * f[:, n:] * (1 if p is None else p.double()[:, None])
    out = R.mm(y, w2, ends)[0]
    dy = R.dgrad(dout, w2, ends)[0]
    dfc1, dp, y2, _ = R.swiglu_bwd(dy, f if fc1 is None else fc1, p)
    E = w1.shape[0]
    return (out, R.dgrad(dfc1, w1, ends)[0], dp, R.wgrad(dfc1, x, ends, E)[0], R.wgrad(dout, y2, ends, E)[0])


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


CASES = [([130, 0, 257, 33], 9, 264, 136), ([1, 2, 0, 1], 0, 72, 40), ([0, 600], 0, 512, 320), ([64, 64], 64, 128, 8)]


@pytest.mark.parametrize("counts,tail,H,n", CASES)
@pytest.mark.parametrize("checkpoint", ["fp8", "bf16"])
@pytest.mark.parametrize("probs", [True, False])
def test_module_against_64_bits(sw, counts, tail, H, n, checkpoint, probs):
    from gate_up_swiglu_gb300.experts import ExpertsSwiGLU, group_ends

    x, w1, w2, p, dout, c = _inputs(counts, tail, H, n, H + n, probs)
    ends = group_ends(c)
    m = ExpertsSwiGLU(len(counts), H, n, checkpoint=checkpoint, device="cuda")
    with torch.no_grad():
        m.w1.copy_(w1), m.w2.copy_(w2)
        plain = m(x, c, p)
    xg = x.clone().requires_grad_(True)
    pg = None if p is None else p.clone().requires_grad_(True)
    out = m(xg, c, pg)
    assert torch.equal(out, plain), "keeping a checkpoint must not change the forward"
    out.backward(dout)
    fc1 = None
    if checkpoint == "fp8":
        _, q, scales = sw.swiglu_grouped_fc1_fwd(x, w1, ends, p, save="fp8")
        fc1 = R.restored(q, scales)
    got = (out.detach(), xg.grad, None if pg is None else pg.grad, m.w1.grad, m.w2.grad)
    ref = _reference(x, w1, w2, p, dout, ends, fc1)
    true = _reference(x, w1, w2, p, dout, ends)
    for name, a, b, t in zip(("out", "dx", "dprobs", "dw1", "dw2"), got, ref, true):
        if a is None:
            continue
        assert _rel(a, b) < 1e-2, name
        assert _rel(a, t) < (0.1 if checkpoint == "fp8" else 1e-2), name
    live = sum(counts)
    for t in (out, xg.grad) + ((pg.grad,) if pg is not None else ()):
        assert live == t.shape[0] or float(t[live:].detach().abs().max()) == 0.0
    for e, k in enumerate(counts):
        if k == 0:
            assert float(m.w1.grad[e].abs().max()) == 0.0 and float(m.w2.grad[e].abs().max()) == 0.0
    assert sw.grouped_timeout_flag() == 0


def test_backward_twice_and_frozen_parts(sw):
    """retain_graph gives the same gradients again (nothing kept is written over);
    a frozen weight gets no gradient and changes no other."""
    from gate_up_swiglu_gb300.experts import ExpertsSwiGLU

    x, w1, w2, p, dout, c = _inputs([40, 7, 90], 3, 136, 72, 5)
    m = ExpertsSwiGLU(3, 136, 72, device="cuda")
    xg = x.clone().requires_grad_(True)
    out = m(xg, c, p)
    first = torch.autograd.grad(out, (xg, m.w1, m.w2), dout, retain_graph=True)
    again = torch.autograd.grad(out, (xg, m.w1, m.w2), dout)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    m.w2.requires_grad_(False)
    (dw1,) = torch.autograd.grad(m(x, c, p), (m.w1,), dout)
    assert torch.equal(dw1, first[1])


def test_checkpoint_is_small(sw):
    """Training memory: with the 8-bit checkpoint the layer holds about half the
    bytes of the bf16 one between forward and backward."""
    from gate_up_swiglu_gb300.experts import ExpertsSwiGLU

    held = {}
    for kind in ("fp8", "bf16"):
        m = ExpertsSwiGLU(2, 128, 4096, checkpoint=kind, device="cuda")
        x = torch.randn(4096, 128, device="cuda").bfloat16().requires_grad_(True)
        c = torch.tensor([2000, 2096], device="cuda")
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = m(x, c)
        held[kind] = torch.cuda.memory_allocated() - before - out.numel() * 2
        del out
    n, rows = 4096, 4096
    assert held["bf16"] >= 4 * n * rows and held["fp8"] <= (2 * n + n // 16) * rows * 1.05 + (1 << 20)


def test_fp8_input_store_of_the_activation_modules(sw):
    from gate_up_swiglu_gb300.autograd import GateUpSwiGLU, WeightedGateUpSwiGLU
    from gate_up_swiglu_gb300.experts import ckpt8_swiglu

    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, 5, 2 * 72, generator=g, device="cuda").bfloat16()
    w = torch.rand(30, 1, generator=g, device="cuda", dtype=torch.float32)
    dy = torch.randn(6, 5, 72, generator=g, device="cuda").bfloat16()
    a, b = x.clone().requires_grad_(True), x.clone().requires_grad_(True)
    y = GateUpSwiGLU(native_fp8=True)(a, None, True)
    assert torch.equal(y, sw.swiglu_gateup_fwd(x))
    y.backward(dy)
    ckpt8_swiglu(b).backward(dy)
    assert torch.equal(a.grad, b.grad)
    _, q, s = sw.swiglu_ckpt8_fwd(x)
    assert torch.equal(a.grad, sw.swiglu_ckpt8_bwd(dy, q, s)[0])
    x2, wg = x.view(30, 144).clone().requires_grad_(True), w.bfloat16().requires_grad_(True)
    y = WeightedGateUpSwiGLU(native_fp8=True)(x2, None, wg, True)
    y.backward(dy.view(30, 72))
    dx, dw, _ = sw.swiglu_ckpt8_bwd(dy.view(30, 72), q.view(30, 144), s.view(30, -1), wg.detach().float().view(-1))
    assert torch.equal(x2.grad, dx) and torch.equal(wg.grad, dw.view(30, 1).bfloat16())
