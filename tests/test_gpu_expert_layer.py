"""The differentiable expert layer, and the example that trains and serves it."""
import importlib.util
import os

import pytest
import torch

from dense_fp32_gemm_gb300.layers import expert_linear

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_gradients_are_those_of_the_plain_layer():
    """FP32, against the same layer in 64 bits: each value is a sum of at most
    64 products, so off by less than 2^-16 of the sum of magnitudes."""
    g = torch.Generator().manual_seed(1)
    x0, w0, dy = (torch.randn(s, generator=g).cuda() for s in [(40, 64), (3, 24, 64), (40, 24)])
    off = torch.tensor([0, 13, 13, 40], dtype=torch.int32, device="cuda")
    x, w = x0.clone().requires_grad_(), w0.clone().requires_grad_()
    y = expert_linear(x, w, off)
    y.backward(dy)
    xd, wd = x0.double().requires_grad_(), w0.double().requires_grad_()
    yd = torch.cat([xd[:13] @ wd[0].T, xd[13:] @ wd[2].T])
    yd.backward(dy.double())
    for got, want in ((y.detach(), yd.detach()), (x.grad, xd.grad), (w.grad, wd.grad)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -16 * (64 + want.abs())).all())
    assert bool((w.grad[1] == 0).all())


def test_example_learns_and_serves():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms, error = example.run(tokens=300, experts=5, width=136, steps=15)
    assert losses[-1] < 0.9 * losses[0]
    assert all(0.0 < n < 100.0 for n in norms)
    # two roundings to 8 bits, each off by at most half a step of 1/127 of a row's
    # largest value (some four times its root mean square)
    assert error < 0.03
