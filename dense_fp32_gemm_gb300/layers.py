"""The linear layer of a set of experts as torch autograd sees it: the three
grouped products of binding.py behind one function."""
from __future__ import annotations

import torch

from . import binding


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, offsets):
        ctx.save_for_backward(x, weight, offsets)
        return binding.grouped_gemm(x, weight, offsets, op="T")

    @staticmethod
    def backward(ctx, dy):
        x, weight, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = binding.grouped_gemm(dy, weight, offsets, op="N") if ctx.needs_input_grad[0] else None
        dw = binding.grouped_wgrad(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def expert_linear(x, weight, offsets):
    """y[r] = x[r] @ weight[e].T for the rows r of expert e, offsets[e] <= r <
    offsets[e + 1]; weight is (E, N, K), offsets E + 1 int32 bounds on the
    device that cover every row of x. Differentiable in x and weight."""
    return _ExpertLinear.apply(x, weight, offsets)
