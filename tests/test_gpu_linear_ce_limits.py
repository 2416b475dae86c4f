"""The loss over a vocabulary where its contract ends: infinite operands.

Tolerances. The logits of 16-bit operands leave the tensor cores, which truncate, every
512 products, that is 32 instructions: off by at most 32 * 2^-23 < 4e-6 of the sum of
magnitudes S, the loss, of two logits, by 8e-6 S."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from test_gpu_linear_ce import formula, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def masked(dtype):
    """A word whose logit is -infinity for every token, by one column."""
    x, w, target = inputs(90, 600, 64, dtype, ignored=0.0)
    target[target == 599] = 0
    x[:, 63] = 1.0
    w[599, 63] = float("-inf")
    return x, w, target


@pytest.mark.parametrize("rows", [90, 20])              # tokens on the lanes, and words
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_words_of_minus_infinity(dtype, rows):
    x, w, target = masked(dtype)
    x, target = x[:rows], target[:rows]
    loss, lse = B.linear_cross_entropy(x, w, target)
    ref_loss, ref_lse, s = formula(x, w[:599], target)
    assert bool(((lse.double() - ref_lse).abs() <= 4e-6 * s + 2e-6 + ref_lse.abs() * 2 * U).all())
    assert bool(((loss.double() - ref_loss).abs() <= 8e-6 * s + 2e-6 + ref_lse.abs() * 4 * U).all())
    # all words but one
    w[:599, 63] = float("-inf")
    w[599, 63] = 0
    target[:] = 599
    assert bool((B.linear_cross_entropy(x, w, target)[0].abs() <= 2e-6 + 8e-6 * s).all())
    # none left: the logarithm of 0
    w[599, 63] = float("-inf")
    assert bool((B.linear_cross_entropy(x, w, target)[1] == float("-inf")).all())


def test_infinite_fp32_operands_give_nan():
    """Cut into three parts they are no numbers any more, as in the grouped products."""
    x, w, target = masked(torch.float32)
    loss, lse = B.linear_cross_entropy(x, w, target)
    assert bool(loss.isnan().all()) and bool(lse.isnan().all())
    x, w, target = inputs(90, 600, 64, torch.float32, ignored=0.0)
    clean = B.linear_cross_entropy(x, w, target)
    for bad in (float("inf"), float("-inf"), float("nan")):
        x[17, 5] = bad
        loss, lse = B.linear_cross_entropy(x, w, target)
        others = torch.arange(90, device="cuda") != 17
        assert bool(loss[17].isnan()) and bool(lse[17].isnan())
        assert torch.equal(loss[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    # the largest numbers are no infinities
    x, w = torch.full((3, 8), 3e38, device="cuda"), torch.zeros(40, 8, device="cuda")
    w[7] = 2.0 ** -126
    loss, lse = B.linear_cross_entropy(x, w, torch.full((3,), 7, device="cuda"))
    z = 8 * x[0, 0].double() * 2.0 ** -126
    want = (z.exp() + 39).log()
    assert bool(((lse.double() - want).abs() <= 2e-6 + 2.0 ** -20 * z).all())
