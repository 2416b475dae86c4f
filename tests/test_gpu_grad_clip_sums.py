"""Sums of squares that FP32 cannot hold.

Squares are summed in FP32 over at most 32 values, whatever the piece a
thread takes (a list of 64 MB and more takes twice as many vectors).

The first value a thread adds is 1, the others' squares are half an ulp of 1,
which round away (ties to even) for as long as they meet it in FP32. With n
values in one FP32 sum the sum loses (n - 1) * 2^-24 of 1, so a norm that keeps
to 32 is at most 31 / 2 * 2^-24 too small, and 20 * 2^-24 hold it with the
rounding to FP32."""
import math

import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("numel", [1 << 20, 1 << 25, (1 << 25) + 4096 + 5])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vecs", [4, 8])
def test_norm_of_values_that_round_away(numel, t, vecs):
    per = 16 // t.itemsize
    piece = vecs * 256 * per                       # values of a piece of that many vectors a thread
    g = torch.full((-(-numel // piece) * piece,), 2.0 ** -12, device="cuda").to(t)
    g.view(-1, vecs, 256, per)[:, 0, :, 0] = 1.0   # first value of every thread's share
    g = g[:numel].clone()
    want = math.sqrt(sum(float(c.double().square().sum()) for c in g.split(1 << 24)))
    norm = float(B.clip_grad_norm([g], 1e9))
    assert abs(norm - want) <= 20 * 2.0 ** -24 * want


@pytest.mark.parametrize("t,value", [(torch.float32, 1e-24), (torch.float32, 1e-38), (torch.float32, 2.0 ** -149),
                                     (torch.bfloat16, 1e-30), (torch.float32, 1e-15)])
@pytest.mark.parametrize("numel", [1, 5, 5000, 1 << 25])
@pytest.mark.parametrize("zeros", [False, True])
def test_norm_of_values_whose_squares_vanish(t, value, numel, zeros):
    """Squares below FP32's range count all the same, between zeros too."""
    g = torch.full((numel,), value, device="cuda").to(t)
    if zeros:
        g.view(-1)[: numel // 2] = -0.0
    want = math.sqrt(float(g.double().square().sum()))
    norm = float(B.clip_grad_norm([g], 1e9))
    # (a subnormal norm is rounded to FP32's last place)
    assert abs(norm - want) <= 20 * 2.0 ** -24 * want + 2.0 ** -150


def test_norm_of_zeros():
    for numel in (3, 10000, 1 << 25):
        assert float(B.clip_grad_norm([torch.zeros(numel, device="cuda")], 1.0)) == 0.0
