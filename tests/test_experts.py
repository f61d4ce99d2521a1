"""Policy of the experts' layer and of the opt-in fp8 input storage that needs no GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def mods():
    from conftest import build_library

    build_library()
    from gate_up_swiglu_gb300 import autograd, experts

    return autograd, experts


def test_experts_refusals(mods):
    _, ex = mods
    with pytest.raises(ValueError, match="checkpoint"):
        ex.ExpertsSwiGLU(2, 16, 8, checkpoint="int4")
    m = ex.ExpertsSwiGLU(2, 16, 8)
    with pytest.raises(ValueError, match="counts"):
        m(torch.zeros(4, 16).bfloat16(), torch.tensor([1, 2, 1]))
    with pytest.raises(ValueError, match="rows"):
        m(torch.zeros(2, 2, 16).bfloat16(), torch.tensor([1, 3]))
    with pytest.raises(ValueError, match="CUDA"):
        m(torch.zeros(4, 16).bfloat16(), torch.tensor([1, 3]))
    with pytest.raises(ValueError, match="checkpoint"):
        ex.ExpertsSwiGLUFunction.apply(torch.zeros(4, 16), None, m.w1, m.w2, torch.zeros(2), "int4")


def test_group_ends(mods):
    _, ex = mods
    ends = ex.group_ends(torch.tensor([3, 0, 5]))
    assert ends.dtype == torch.int32 and ends.tolist() == [3, 3, 8]


def test_native_fp8_takes_the_input_without_a_bias_only(mods):
    ag, _ = mods
    m = ag.GateUpSwiGLU(native_fp8=True, native_bias=True)
    with pytest.raises(ValueError, match="CUDA"):  # on its way to the kernels
        m(torch.zeros(4, 8), None, True)
    with pytest.raises(NotImplementedError, match="fp8_input_store"):
        m(torch.zeros(4, 8), torch.zeros(8), True)
    with pytest.raises(NotImplementedError, match="cpu_offload_input"):
        m(torch.zeros(4, 8), None, True, True)
    w = ag.WeightedGateUpSwiGLU(native_fp8=True)
    with pytest.raises(NotImplementedError, match="fp8_input_store"):
        w(torch.zeros(4, 8), torch.zeros(8), torch.ones(4), True)
    with pytest.raises(ValueError, match="one value per row"):
        w(torch.zeros(4, 8), None, torch.ones(3), True)
    with pytest.raises(ValueError, match="CUDA"):
        w(torch.zeros(4, 8), None, torch.ones(4), True)


def test_counts_of_two_dimensions_are_summed_over_all(mods):
    """Not along the first one only, which leaves [[3, 0, 5]] as it is."""
    _, ex = mods
    for shape in ((1, 3), (3, 1), (3,)):
        ends = ex.group_ends(torch.tensor([3, 0, 5]).view(shape))
        assert ends.dtype == torch.int32 and ends.tolist() == [3, 3, 8]


def test_a_second_derivative_is_refused(mods, monkeypatch):
    """The backward's kernels are no differentiable operations: a gradient taken with
    create_graph must not pass for a constant.  (Stand-ins for the kernels: no GPU.)"""
    _, ex = mods
    like = torch.zeros_like
    for name, fn in dict(
            swiglu_ckpt8_fwd=lambda x, w: (x[..., ::2] * 1, like(x), like(x)),
            swiglu_ckpt8_bwd=lambda dy, q, s, w, return_y=False: (torch.cat([dy, dy], -1), w, like(dy)),
            swiglu_grouped_fc1_fwd=lambda x, w, e, p, save=None: (x.new_ones(x.shape[0], w.shape[1] // 2), like(x), like(x)),
            swiglu_grouped_mm_fwd=lambda x, w, e: x.new_ones(x.shape[0], w.shape[1]),
            swiglu_grouped_mm_dgrad=lambda dy, w, e: dy.new_ones(dy.shape[0], w.shape[2]),
            swiglu_grouped_mm_wgrad=lambda dy, x, e, dtype: dy.new_ones(2, dy.shape[1], x.shape[1])).items():
        monkeypatch.setattr(ex, name, fn)
    x = torch.ones(4, 8, requires_grad=True)
    w1, w2 = torch.ones(2, 12, 8, requires_grad=True), torch.ones(2, 8, 6, requires_grad=True)
    for y in (ex.ckpt8_swiglu(x, torch.ones(4, requires_grad=True)),
              ex.ExpertsSwiGLUFunction.apply(x, None, w1, w2, torch.tensor([2, 4]))):
        (dx,) = torch.autograd.grad((y * y).sum(), (x,), create_graph=True)
        assert dx.shape == x.shape
        with pytest.raises(RuntimeError, match="once_differentiable"):
            ((dx * dx).sum() + (x * x).sum()).backward()
