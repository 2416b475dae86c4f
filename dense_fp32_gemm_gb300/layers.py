"""The linear layer of a set of experts as torch autograd sees it: the three
grouped products of binding.py behind one function. Each product's gradients
are products of the same kinds, so derivatives of any order come out."""
from __future__ import annotations

import torch

from . import binding


def _flip(op):
    return "N" if op == "T" else "T"


class _Rows(torch.autograd.Function):
    """y[r] = x[r] op(w[e])."""

    @staticmethod
    def forward(ctx, x, w, offsets, op):
        ctx.save_for_backward(x, w, offsets)
        ctx.op = op
        return binding.grouped_gemm(x, w, offsets, op=op)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = _Rows.apply(dy, w, offsets, _flip(ctx.op)) if ctx.needs_input_grad[0] else None
        dw = None
        if ctx.needs_input_grad[1]:
            a, b = (dy, x) if ctx.op == "T" else (x, dy)
            dw = _Weights.apply(a, b, offsets)
        return dx, dw, None, None


class _Weights(torch.autograd.Function):
    """c[e] = a_e.T b_e over the rows of each group."""

    @staticmethod
    def forward(ctx, a, b, offsets):
        ctx.save_for_backward(a, b, offsets)
        return binding.grouped_wgrad(a, b, offsets)

    @staticmethod
    def backward(ctx, dc):
        a, b, offsets = ctx.saved_tensors
        dc = dc.contiguous()
        da = _Rows.apply(b, dc, offsets, "T") if ctx.needs_input_grad[0] else None
        db = _Rows.apply(a, dc, offsets, "N") if ctx.needs_input_grad[1] else None
        return da, db, None


def expert_linear(x, weight, offsets):
    """y[r] = x[r] @ weight[e].T for the rows r of expert e, offsets[e] <= r <
    offsets[e + 1]; weight is (E, N, K), offsets E + 1 int32 bounds on the
    device that cover every row of x. Differentiable in x and weight, any
    number of times."""
    return _Rows.apply(x, weight, offsets, "T")
