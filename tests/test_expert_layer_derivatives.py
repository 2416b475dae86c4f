"""Second derivatives of expert_linear. On the CPU the three products are
replaced by plain ones, in 64 bits, so that what is tested is the graph; on the
GPU the kernels run."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding, layers


def parts(offsets):
    b = offsets.tolist()
    return [(e, slice(b[e], b[e + 1])) for e in range(len(b) - 1)]


def plain_rows(x, w, offsets, op="T"):
    out = torch.cat([x[r] @ (w[e].mT if op == "T" else w[e]) for e, r in parts(offsets)])
    return out


def plain_gemm(X, W, offsets, op="T", **_):
    with torch.no_grad():            # as the library's call: no graph
        return plain_rows(X, W, offsets, op)


def plain_wgrad(A, B, offsets, **_):
    with torch.no_grad():
        return torch.stack([A[r].mT @ B[r] for _, r in parts(offsets)])


def case(device, t):
    g = torch.Generator().manual_seed(3)
    x, w, v = (torch.randn(s, generator=g, dtype=torch.float64).to(t).to(device) for s in [(9, 6), (3, 5, 6), (9, 5)])
    off = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device=device)
    return x.requires_grad_(), w.requires_grad_(), v, off


def penalty(layer, x, w, v, off):
    """A loss with a gradient in it: its derivatives need the second ones of the layer."""
    y = layer(x, w, off)
    loss = (torch.tanh(y) * v).sum()
    dx, dw = torch.autograd.grad(loss, [x, w], create_graph=True)
    return loss + dx.square().sum() + (dw ** 3).sum()


def test_graph_of_the_second_derivatives(monkeypatch):
    monkeypatch.setattr(binding, "grouped_gemm", plain_gemm)
    monkeypatch.setattr(binding, "grouped_wgrad", plain_wgrad)
    x, w, v, off = case("cpu", torch.float64)
    got = torch.autograd.grad(penalty(layers.expert_linear, x, w, v, off), [x, w])
    want = torch.autograd.grad(penalty(plain_rows, x, w, v, off), [x, w])
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    assert torch.autograd.gradcheck(lambda x, w: layers.expert_linear(x, w, off), (x, w))
    assert torch.autograd.gradgradcheck(lambda x, w: layers.expert_linear(x, w, off), (x, w))


def test_what_needs_no_gradient_gets_none(monkeypatch):
    monkeypatch.setattr(binding, "grouped_gemm", plain_gemm)
    monkeypatch.setattr(binding, "grouped_wgrad", plain_wgrad)
    x, w, v, off = case("cpu", torch.float64)
    y = layers.expert_linear(x.detach(), w, off)
    dw, = torch.autograd.grad((y * v).sum(), [w], create_graph=True)
    assert torch.allclose(dw, plain_wgrad(v, x, off)) and not dw.requires_grad
    y = layers.expert_linear(x, w.detach(), off)
    dx, = torch.autograd.grad((y * v).sum(), [x])
    assert torch.allclose(dx, plain_gemm(v, w, off, op="N"))


@pytest.mark.gpu
def test_second_derivatives_of_the_kernels():
    """FP32 against 64 bits: sums of at most 9 products of values that are themselves off by some
    1e-6 of magnitudes below 100, through three layers of products."""
    x, w, v, off = case("cuda", torch.float32)
    got = torch.autograd.grad(penalty(layers.expert_linear, x, w, v, off), [x, w])
    x, w, v, off = case("cuda", torch.float64)
    want = torch.autograd.grad(penalty(plain_rows, x, w, v, off), [x, w])
    for a, b in zip(got, want):
        assert float((a.double() - b).norm() / b.norm()) < 1e-4
