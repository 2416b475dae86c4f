"""sgemm_grad_clip against sums in 64 bits.

Tolerance of the norm: at most 32 squares are added in FP32 (33 * 2^-24
relative on their sum, halved by the root), the rest in FP64, and the result is
rounded to FP32: 20 * 2^-24 relative. The outputs: the coefficient's error plus
two roundings of FP32 and one of the output type.
"""
import math

import numpy as np
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
NORM_TOL = 20 * 2.0 ** -24


def make(sizes, t, seed, scale=1.0, shift=0):
    """Tensors one behind the other in one buffer, `shift` elements into it,
    with a guard of NaN on both sides."""
    g = torch.Generator().manual_seed(seed)
    n = sum(sizes)
    store = torch.full((n + shift + 64,), float("nan"), dtype=t, device="cuda")
    store[shift: shift + n] = (torch.randn((n,), generator=g) * scale).to(t).cuda()
    return store, list(store[shift: shift + n].split(sizes))


def check(grads, max_norm, out=None):
    before = [g.clone() for g in grads]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    coef = min(1.0, max_norm / (want + 1e-6))
    norm = B.clip_grad_norm(grads, max_norm, out=out)
    assert abs(float(norm) - want) <= NORM_TOL * want
    for o, b in zip(grads if out is None else out, before):
        if coef == 1.0:
            assert torch.equal(o, b)
            continue
        ref = b.double() * coef
        tol = (NORM_TOL + 4 * 2.0 ** -24 + ROUND[o.dtype]) * ref.abs() + (2.0 ** -24 if o.dtype == torch.float16 else 1e-38)
        assert bool(((o.double() - ref).abs() <= tol).all())
    if out is not None:
        for g, b in zip(grads, before):
            assert torch.equal(g, b)


SIZES = [[1], [7, 1, 3], [4096], [4097, 1, 8191, 0, 16385], [100000, 3, 250001], [1] * 70]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_in_place_and_out_of_place(t, sizes, shift):
    store, grads = make(sizes, TYPES[t], 1, shift=shift)
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    ostore, out = make(sizes, TYPES[t], 2, shift=2)
    check(grads, 0.25 * norm, out=out)
    check(grads, 4.0 * norm, out=out)      # not clipped: copied
    check(grads, 4.0 * norm)               # not clipped, in place
    check(grads, 0.25 * norm)
    for s, k in ((store, shift), (ostore, 2)):
        n = sum(sizes)
        assert bool(s[:k].isnan().all()) and bool(s[k + n:].isnan().all())


def test_mixed_types_and_many_tensors():
    rng = np.random.default_rng(1)
    grads = []
    for i in range(2300):                  # three lists
        t = list(TYPES.values())[i % 3]
        grads.append(torch.randn(int(rng.integers(1, 600))).to(t).cuda())
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    check(grads, 0.1 * norm)
    check(grads, 10.0 * norm)


def test_norm_only_and_empty():
    _, grads = make([1000, 5], torch.float32, 3)
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm = torch.empty((), device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert B.sgemm_grad_clip([g.data_ptr() for g in grads], None, [g.numel() for g in grads], [0, 0], 1.0,
                             norm.data_ptr(), s) == 0
    assert abs(float(norm) - want) <= NORM_TOL * want
    for n, sizes in ((0, []), (2, [0, 0])):
        norm.fill_(-1.0)
        assert B.sgemm_grad_clip([0] * n, [0] * n, sizes, [0] * n, 1.0, norm.data_ptr(), s) == 0
        assert float(norm) == 0.0


def test_extremes():
    def one(values, max_norm, t=torch.float32):
        g = torch.tensor(values, dtype=t, device="cuda")
        n = B.clip_grad_norm([g], max_norm)
        return float(n), g.cpu().tolist()

    n, g = one([3e25, -4e25], 5.0)                     # squares beyond FP32
    assert abs(n - 5e25) < 1e-6 * 5e25 and abs(g[0] - 3.0) < 1e-5 and abs(g[1] + 4.0) < 1e-5
    n, g = one([3e-19, 4e-19], 1.0)                    # squares below its normal range
    assert abs(n - 5e-19) < 1e-6 * 5e-19 and g == torch.tensor([3e-19, 4e-19]).tolist()
    n, g = one([0.0, -0.0], 1.0)
    assert n == 0.0 and g == [0.0, 0.0]
    n, g = one([1.0, float("inf")], 1.0)
    assert n == float("inf") and g[0] == 0.0 and math.isnan(g[1])
    n, g = one([1.0, float("nan")], 1.0)
    assert math.isnan(n) and math.isnan(g[0]) and math.isnan(g[1])
    n, g = one([3.0, 4.0], 0.0)
    assert n == 5.0 and g == [0.0, 0.0]
    n, g = one([3.0, 4.0], float("inf"))
    assert n == 5.0 and g == [3.0, 4.0]


def test_large_tensor_same_bits():
    g = torch.randn(30_000_001, device="cuda").bfloat16()
    out = torch.empty_like(g)
    norms = [float(B.clip_grad_norm([g], 1.0, out=[out])) for _ in range(4)]
    assert len(set(norms)) == 1
    want = float(g.double().square().sum().sqrt())
    assert abs(norms[0] - want) <= NORM_TOL * want


def test_graph():
    _, grads = make([5000, 77], torch.float32, 5)
    out = [torch.empty_like(g) for g in grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.clip_grad_norm(grads, 1.0, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            norm = B.clip_grad_norm(grads, 1.0, out=out)
        grads[0].mul_(3.0)
        graph.replay()
    s.synchronize()
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - want) <= NORM_TOL * want
