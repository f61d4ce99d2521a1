"""The dense MLP sublayer's modules: the layer norm in front of linear_fc1 (with
its gradients) and the gated MLP with weights and activations in 4 bits.

    norm = LayerNorm(4096, device="cuda")                  # trains and serves
    h = norm(x)                                            # into Fc1SwiGLU, or
    mlp = Mx4SwiGLU.from_weights(fc1.weight, w2)           # serving
    out = x + mlp(h)

While a backward pass is captured into a CUDA graph, no eager graph of the same leaves
may be alive (an output that is still held, say): torch hands a leaf's gradient to the
stream of its first graph, which is not part of the capture, and the capture fails.

All arithmetic runs in the CUDA kernels; this module only decides what to call.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import mx4_scales_shape, swiglu_layer_norm_bwd, swiglu_layer_norm_fwd, swiglu_mx4_quantize
from .autograd import carries_tangent
from .mx4 import MX4_BLOCK, SCALE_DTYPE, _mlp_fwd, _need_scale_type


class LayerNormFunction(torch.autograd.Function):
    """y = (x - mean) rstd weight + bias; weight and bias optional."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor], eps: float):
        y, mean, rstd = swiglu_layer_norm_fwd(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.bias = None if bias is None else (bias.shape, bias.dtype)
        return y

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph
    def backward(ctx, dy: torch.Tensor):
        x, mean, rstd, weight = ctx.saved_tensors
        need_w, need_b = ctx.needs_input_grad[1:3]
        dbias = None
        if need_b:
            dbias = torch.empty(ctx.bias[0], dtype=ctx.bias[1], device=x.device)
        dx, dw, db = swiglu_layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight, bias_grad=need_b, dbias=dbias,
                                           weight_grad=need_w)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """The layer norm over the last dimension; keeps x, mean and rstd where a gradient
    will be asked for.  It has no forward-mode derivative: a tangent raises."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)) or \
            carries_tangent(x, weight, bias):
        return LayerNormFunction.apply(x, weight, bias, eps)
    return swiglu_layer_norm_fwd(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """Layer norm over a last dimension of ``hidden``, with a weight and (``bias``) a
    bias of ``dtype``; the input is of that dtype, or bfloat16 with float32
    parameters."""

    def __init__(self, hidden: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.hidden, self.eps = hidden, eps
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.hidden:
            raise ValueError(f"x must be [..., {self.hidden}]")
        return layer_norm(x, self.weight, self.bias, self.eps)


class Mx4SwiGLU(torch.nn.Module):
    """The gated MLP (bias-free) with weights and activations in 4 bits, for serving:
    w1 [2 * ffn_hidden, hidden] with gate rows first, w2 [out, ffn_hidden] (out =
    hidden unless given), held as uint8 buffers of codes and scale bytes, which a change
    of the module's dtype leaves alone.  It has no derivatives: an input that requires a
    gradient is refused while gradients are on, and so is one with a tangent."""

    def __init__(self, hidden: int, ffn_hidden: int, out: int = None, device=None):
        super().__init__()
        _need_scale_type()
        out = hidden if out is None else out
        self.hidden, self.ffn_hidden = hidden, ffn_hidden
        for name, rows, cols, parts in (("w1", 2 * ffn_hidden, hidden, 2), ("w2", out, ffn_hidden, 1)):
            blocks = (cols + MX4_BLOCK - 1) // MX4_BLOCK
            self.register_buffer(name + "_q", torch.zeros(rows, 16 * blocks, dtype=torch.uint8, device=device))
            scales = torch.zeros(mx4_scales_shape(rows, cols, parts), dtype=torch.uint8, device=device)
            self.register_buffer(name + "_scales", scales)

    @classmethod
    def from_weights(cls, w1: torch.Tensor, w2: torch.Tensor) -> "Mx4SwiGLU":
        """From float32 or bfloat16 weights w1 [2n, hidden] (gate rows first), w2 [out, n]."""
        if w1.dim() != 2 or w2.dim() != 2 or w1.shape[0] != 2 * w2.shape[1]:
            raise ValueError("w1 must be [2n, hidden] and w2 [out, n]")
        mod = cls(w1.shape[1], w2.shape[1], w2.shape[0], device=w1.device)
        swiglu_mx4_quantize(w1.detach(), 2, mod.w1_q, mod.w1_scales.view(SCALE_DTYPE))
        swiglu_mx4_quantize(w2.detach(), 1, mod.w2_q, mod.w2_scales.view(SCALE_DTYPE))
        return mod

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.hidden:
            raise ValueError(f"x must be [..., {self.hidden}]")
        if torch.is_grad_enabled() and x.requires_grad:
            raise NotImplementedError("the 4-bit MLP has no backward: call it under torch.no_grad()")
        if carries_tangent(x):
            raise NotImplementedError("the 4-bit MLP has no forward-mode derivative: call it on the primal tensor")
        return _mlp_fwd(x, self.w1_q, self.w1_scales, self.w2_q, self.w2_scales, None, None, None, torch.uint8)
