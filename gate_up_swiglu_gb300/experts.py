"""The routed experts' MLP as an autograd function and a module: the grouped
products and the 8-bit activation checkpoint run together.

    y[t]   = probs[t] * silu(W1g[e] x[t]) * (W1u[e] x[t])     (swiglu_grouped_fc1_fwd)
    out[t] = W2[e] y[t]                                        (swiglu_grouped_mm_fwd)

Rows are sorted by expert (Megatron's grouped MLP after its token permutation);
``probs`` are the routing weights that ``weighted_bias_swiglu_impl`` applies
between the two products.  What the backward pass keeps besides x and the
weights, per row of n ffn columns:

    checkpoint="fp8"    2 n + n / 16 bytes: the 8-bit checkpoint of the first
                        product.  The backward makes dfc1, dprobs and y from it in
                        one kernel; they carry its rounding (4 significant bits).
    checkpoint="bf16"   4 n bytes: the first product in bf16, as Megatron keeps it.
                        The backward runs the weighted activation kernels on it.

All arithmetic runs in the CUDA kernels; this module only decides what to call.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (swiglu_ckpt8_bwd, swiglu_ckpt8_fwd, swiglu_gateup_bwd, swiglu_gateup_fwd, swiglu_gateup_weighted_bwd,
               swiglu_gateup_weighted_fwd, swiglu_grouped_fc1_fwd, swiglu_grouped_mm_dgrad, swiglu_grouped_mm_fwd,
               swiglu_grouped_mm_wgrad)
from .autograd import carries_tangent

CHECKPOINTS = ("fp8", "bf16")


def group_ends(counts: torch.Tensor) -> torch.Tensor:
    """The `ends` of the grouped products from the rows per expert (in one dimension or
    with others of size one)."""
    return counts.reshape(-1).cumsum(0, dtype=torch.int32)


class Ckpt8SwiGLUFunction(torch.autograd.Function):
    """y = w[row] * silu(x[..., :n]) * x[..., n:] that keeps x in 8 bits for the
    backward (Megatron's fp8_input_store); ``weights`` (one per row, any float
    dtype) optional.  The gradients are those at the checkpointed x."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weights: Optional[torch.Tensor]):
        w32 = None
        if weights is not None:
            w32 = weights.detach().reshape(-1).to(torch.float32).contiguous()
            ctx.w_shape, ctx.w_dtype = weights.shape, weights.dtype
        y, q, scales = swiglu_ckpt8_fwd(x, w32)
        ctx.save_for_backward(q, scales, w32)
        return y

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph
    def backward(ctx, dy: torch.Tensor):
        q, scales, w32 = ctx.saved_tensors
        dx, dw, _ = swiglu_ckpt8_bwd(dy.contiguous(), q, scales, w32)
        return dx, None if dw is None else dw.reshape(ctx.w_shape).to(ctx.w_dtype)


def ckpt8_swiglu(x: torch.Tensor, weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    return Ckpt8SwiGLUFunction.apply(x, weights)


class ExpertsSwiGLUFunction(torch.autograd.Function):
    """(x [rows, H], probs [rows] or None, w1 [E, 2n, H], w2 [E, H, n], ends [E])
    -> out [rows, H].  Rows of no expert give zeros and get zero gradients."""

    @staticmethod
    def forward(ctx, x, probs, w1, w2, ends, checkpoint="fp8"):
        if checkpoint not in CHECKPOINTS:
            raise ValueError(f"checkpoint must be one of {CHECKPOINTS}")
        x, w1, w2 = x.contiguous(), w1.contiguous(), w2.contiguous()
        p32 = None
        if probs is not None:
            p32 = probs.detach().reshape(-1).to(torch.float32).contiguous()
            ctx.p_shape, ctx.p_dtype = probs.shape, probs.dtype
        y, *kept = swiglu_grouped_fc1_fwd(x, w1, ends, p32, save=checkpoint)
        out = swiglu_grouped_mm_fwd(y, w2, ends)
        ctx.save_for_backward(x, p32, w1, w2, ends, *kept)
        ctx.checkpoint = checkpoint
        return out

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph
    def backward(ctx, dout):
        x, p32, w1, w2, ends, *kept = ctx.saved_tensors
        need_x, need_p, need_w1, need_w2 = ctx.needs_input_grad[:4]
        dout = dout.contiguous()
        dx = dprobs = dw1 = dw2 = None
        dy = swiglu_grouped_mm_dgrad(dout, w2, ends)
        if ctx.checkpoint == "fp8":
            dfc1, dp, y = swiglu_ckpt8_bwd(dy, *kept, p32, return_y=need_w2)
        else:
            (fc1,) = kept
            if p32 is not None:
                y = swiglu_gateup_weighted_fwd(fc1, p32) if need_w2 else None
                dfc1, dp = swiglu_gateup_weighted_bwd(dy, fc1, p32)
            else:
                y = swiglu_gateup_fwd(fc1) if need_w2 else None
                dfc1, dp = swiglu_gateup_bwd(dy, fc1), None
        del dy
        if need_w2:
            dw2 = swiglu_grouped_mm_wgrad(dout, y, ends, dtype=w2.dtype)
        if need_w1:
            dw1 = swiglu_grouped_mm_wgrad(dfc1, x, ends, dtype=w1.dtype)
        if need_x:
            dx = swiglu_grouped_mm_dgrad(dfc1, w1, ends)
        if need_p and dp is not None:
            dprobs = dp.reshape(ctx.p_shape).to(ctx.p_dtype)
        return dx, dprobs, dw1, dw2, None, None


class ExpertsSwiGLU(torch.nn.Module):
    """The experts of an MoE layer (bias-free): w1 [E, 2 * ffn_hidden, hidden] with
    gate rows first, w2 [E, hidden, ffn_hidden].

    forward(x [rows, hidden], counts [E], probs=None): rows sorted by expert,
    ``counts`` the rows per expert (a CUDA integer tensor; the host does not read
    it), ``probs`` one routing weight per row.  Without gradients nothing is kept
    of the first product (prefill and decode steps).  There is no forward-mode derivative:
    a tangent raises."""

    def __init__(self, experts: int, hidden: int, ffn_hidden: int, checkpoint: str = "fp8", device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        if checkpoint not in CHECKPOINTS:
            raise ValueError(f"checkpoint must be one of {CHECKPOINTS}")
        self.checkpoint = checkpoint
        self.w1 = torch.nn.Parameter(torch.empty(experts, 2 * ffn_hidden, hidden, device=device, dtype=dtype))
        self.w2 = torch.nn.Parameter(torch.empty(experts, hidden, ffn_hidden, device=device, dtype=dtype))
        torch.nn.init.normal_(self.w1, std=hidden ** -0.5)
        torch.nn.init.normal_(self.w2, std=ffn_hidden ** -0.5)

    def forward(self, x: torch.Tensor, counts: torch.Tensor, probs: Optional[torch.Tensor] = None) -> torch.Tensor:
        if x.dim() != 2 or counts.numel() != self.w1.shape[0]:
            raise ValueError("x must be [rows, hidden] and counts hold the rows of each expert")
        ends = group_ends(counts)
        tracked = (x, self.w1, self.w2) if probs is None else (x, probs, self.w1, self.w2)
        if torch.is_grad_enabled() and any(t.requires_grad for t in tracked) or carries_tangent(*tracked):
            return ExpertsSwiGLUFunction.apply(x, probs, self.w1, self.w2, ends, self.checkpoint)
        p32 = None if probs is None else probs.reshape(-1).to(torch.float32).contiguous()
        y = swiglu_grouped_fc1_fwd(x.contiguous(), self.w1, ends, p32)
        return swiglu_grouped_mm_fwd(y, self.w2, ends)
