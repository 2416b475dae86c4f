"""The loss over a vocabulary where its contract ends or is tightest: infinite operands,
the exactness of the logits of 16-bit operands, gradients of saturated rows.

Tolerances. The logits of 16-bit operands leave the tensor cores, which truncate, every
512 products, that is 32 instructions: off by at most 32 * 2^-23 < 4e-6 of the sum of
magnitudes S, the loss, of two logits, by 8e-6 S. In the 2-norm n truncations in an
accumulation make 1.4e-8 n of a logit, so an error of E = 32 * 1.4e-8 here; the loss
has that of its target's logit z and that of lse, which moves by the mean of the logits'
own under the softmax: together E * (|z| + sum p |z|). FP32 beside it: lse and loss
between 8 and 16 are rounded to steps of 2^-20 (each 0.29 of one in the 2-norm) and
the exponentials are off by 2^-22: below 6e-7 together."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from test_gpu_linear_ce import formula, inputs, rand, rounding

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,v", [(1024, 16384), (48, 16384)])
def test_exactness_of_the_loss(dtype, t, v):
    x, w, target = inputs(t, v, 2048, dtype, ignored=0.0)
    loss, lse = B.linear_cross_entropy(x, w, target)
    ref_loss, ref_lse, s = formula(x, w, target)
    assert bool(((lse.double() - ref_lse).abs() <= 4e-6 * s + 2e-6 + ref_lse.abs() * 2 * U).all())
    assert bool(((loss.double() - ref_loss).abs() <= 8e-6 * s + 2e-6 + ref_lse.abs() * 4 * U).all())
    z = x.double() @ w.double().mT
    mean = ((z - ref_lse[:, None]).exp() * z.abs()).sum(dim=1)
    off = (loss.double() - ref_loss).square().mean().sqrt()
    most = 32 * 1.4e-8 * (z.gather(1, target[:, None])[:, 0].abs() + mean).square().mean().sqrt() + 6e-7
    assert float(off) <= float(most), (float(off), float(most))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t", [200, 30])
def test_gradients_of_large_logits(dtype, t):
    """Logits of some 10^3, multiples of 64: one word has all of the probability, or some have equal shares. Logits and
    lse are exact but for lse's rounding, so G is off by its own rounding and 3e-6 + lse 2^-23 of the probabilities."""
    v, h = 900, 128
    g = torch.Generator(device="cuda").manual_seed(t)
    x = 64.0 * torch.randint(-1, 2, (t, h), generator=g, device="cuda")
    w = torch.randint(-1, 2, (v, h), generator=g, device="cuda")
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    target[::9] = -100
    x, w = x.to(dtype), w.to(dtype)
    target[1] = int((x[1].double() @ w.double().mT).argmax())       # the word that has it
    d = rand(t, seed=9)
    loss, lse = B.linear_cross_entropy(x, w, target)
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    ref_loss, ref_lse, _, p, grad = formula(x, w, target, d)
    assert float(ref_lse.amax()) > 1000
    assert bool(((loss.double() - ref_loss).abs() <= 2e-6 + ref_lse.abs() * 4 * U).all())
    xd, wd = x.double(), w.double()
    off = torch.finfo(dtype).eps / 2 * grad.abs() + (3e-6 + ref_lse.abs() * 2.0 ** -23)[:, None] * p
    off = off + (float(d.abs().amax()) * 2.0 ** -38 if dtype == torch.float16 else 0.0)
    for got, want, slack in ((dx, grad @ wd, off @ wd.abs() + 1e-5 * (grad.abs() @ wd.abs())),
                             (dw, grad.mT @ xd, off.mT @ xd.abs() + 1e-5 * (grad.abs().mT @ xd.abs()))):
        assert bool(((got.double() - want).abs() <= slack + rounding(want, dtype)).all())
