"""Tensors that a call is given to write count as changed for autograd: a graph
that saved one for its backward pass refuses to use the new values."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu


def calls():
    """name: (call, the tensors it writes, the ones it only reads)"""
    f = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.ones(*s, device="cuda", dtype=torch.int8)  # noqa: E731
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    x, w, y, dy, c = f(4, 8), f(2, 6, 8), f(4, 6), f(4, 6), f(2, 6, 8)
    q, s, qa, qb, sb, z, out = i(4, 8), f(4), i(4, 8), i(6, 8), f(6), f(4, 6), f(4, 8)
    a, b, r = f(4, 5), f(5, 3), f(4, 3)
    return {
        "rows": (lambda: B.grouped_gemm(x, w, off, Y=y), [y], [x, w, off]),
        "wgrad": (lambda: B.grouped_wgrad(dy, x, off, C=c), [c], [dy, x, off]),
        "quantize": (lambda: B.i8_quantize(x, Q=q, scale=s), [q, s], [x]),
        "i8": (lambda: B.i8_gemm(qa, s, qb, sb, C=z), [z], [qa, s, qb, sb]),
        "clip": (lambda: B.clip_grad_norm([x], 1.0, out=[out]), [out], [x]),
        "clip in place": (lambda: B.clip_grad_norm(iter([x, w]), 1.0), [x, w], []),
        "gemm": (lambda: B.gemm(a, b, r, beta=0.0), [r], [a, b]),
    }


@pytest.mark.parametrize("name", ["rows", "wgrad", "quantize", "i8", "clip", "clip in place", "gemm"])
def test_written_tensors_change_their_version(name):
    call, written, read = calls()[name]
    before = [t._version for t in written + read]
    call()
    after = [t._version for t in written + read]
    n = len(written)
    assert all(b < a for b, a in zip(before[:n], after[:n])) and before[n:] == after[n:]


def test_backward_refuses_overwritten_values():
    x, saved = torch.ones(4, 8, device="cuda", requires_grad=True), torch.ones(4, 8, device="cuda")
    loss = (x * saved).sum()
    B.clip_grad_norm([saved], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", ["rows", "wgrad", "quantize", "i8", "clip", "clip in place", "gemm"])
def test_inference_tensors(name):
    with torch.inference_mode():
        call, written, _ = calls()[name]
        call()
        assert all(t.is_inference() for t in written)
