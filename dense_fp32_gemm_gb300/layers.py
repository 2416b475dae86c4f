"""The operators of binding.py as torch autograd sees them.

The linear layer of a set of experts: the three grouped products behind one
function. Each product's gradients are products of the same kinds, so
derivatives of any order come out. The norm and the loss of the output end have
first derivatives; asking for a second raises."""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

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


def _rows(x):
    """x as a matrix of its last dimension's rows (none of them may be there)."""
    return x.reshape(math.prod(x.shape[:-1]), x.shape[-1])


class _Norm(torch.autograd.Function):
    """(y, h) of binding.rms_norm on rows."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, h, rstd = binding.rms_norm(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.with_residual = residual is not None
        return (y, h) if ctx.with_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        dx, dw = dh, None
        if dy is None:              # only h was used
            dw = torch.zeros_like(weight) if need_w else None
        else:
            dx, dw = binding.rms_norm_grad(dy.contiguous(), h, weight, rstd,
                                           dH=None if dh is None else dh.contiguous(),
                                           want=(need_x or need_r, need_w))
        return dx if need_x else None, dw, dx if need_r else None, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """h / sqrt(mean(h^2) + eps) * weight over the last dimension, h = x +
    residual; with a residual (y, h) is returned. Differentiable once in x,
    weight and residual."""
    rows = _rows(x)
    if residual is None:
        return _Norm.apply(rows, weight, None, eps).view(x.shape)
    if residual.shape != x.shape:
        raise ValueError("residual must have the shape of x")
    y, h = _Norm.apply(rows, weight, residual.reshape(rows.shape), eps)
    return y.view(x.shape), h.view(x.shape)


class _CrossEntropy(torch.autograd.Function):
    """binding.linear_cross_entropy's loss of each row."""

    @staticmethod
    def forward(ctx, x, w, target, ignore_index):
        loss, lse = binding.linear_cross_entropy(x, w, target, ignore_index=ignore_index)
        ctx.save_for_backward(x, w, target, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, w, target, lse = ctx.saved_tensors
        dx, dw = binding.linear_cross_entropy_grad(x, w, target, lse, dloss.contiguous(),
                                                   ignore_index=ctx.ignore_index,
                                                   want=ctx.needs_input_grad[:2])
        return dx, dw, None, None


def linear_cross_entropy(x, weight, target, ignore_index=-100, reduction="mean"):
    """Softmax cross entropy of x @ weight.T with the words `target` (int64, the
    leading dimensions of x), without keeping the logits. Rows whose target is
    ignore_index are not counted (but must hold finite numbers). reduction: "mean" over the counted rows (0 if
    there are none), "sum", or "none" (a value a row). Differentiable once in x
    and weight."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError('reduction must be "mean", "sum" or "none"')
    if target.shape != x.shape[:-1]:
        raise ValueError("target must have the leading dimensions of x")
    loss = _CrossEntropy.apply(_rows(x), weight, target.reshape(-1).contiguous(), ignore_index)
    if reduction == "none":
        return loss.view(target.shape)
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (target != ignore_index).sum().clamp(min=1)
