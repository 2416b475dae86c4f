"""How far truncation in the tensor cores may take a sum.

An instruction adds 16 products and truncates the sum it adds to, by less than
2^-23 of it. 16-bit results leave the accumulator every 1024 values of k, 32-bit
results of 16-bit operands every 256; the parts are added with rounding to
nearest (2^-24 of the sum each). So a sum of K products of one sign is short
by less than (64 * 2^-23 + K / 1024 * 2^-24) of itself, or (16 * 2^-23 + K / 256
* 2^-24), whatever K is."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def positive(shape, seed, t, scale):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(shape, generator=g, device="cuda") + 0.5) * scale).to(t)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("k", [4096, 16384, 131072])
@pytest.mark.parametrize("kind", ["rows", "wgrad"])
def test_long_sums_of_one_sign_are_not_short(kind, t, k):
    """16-bit results: rounding is monotone, so a result lies between the rounded ends of the sum's interval."""
    t = TYPES[t]
    off = torch.tensor([0, k if kind == "wgrad" else 256], dtype=torch.int32, device="cuda")
    if kind == "rows":
        x, w = positive((256, k), 1, t, 1 / 64), positive((1, 512, k), 2, t, 1.0)
        got, ref = B.grouped_gemm(x, w, off), x.double() @ w[0].double().mT
    else:
        a, b = positive((k, 520), 1, t, 1 / 64), positive((k, 264), 2, t, 1.0)
        got, ref = B.grouped_wgrad(a, b, off)[0], a.double().mT @ b.double()
    assert got.dtype == t
    short, rounded = 64 * 2.0 ** -23 + k / 1024 * 2.0 ** -24, k / 1024 * 2.0 ** -24
    assert bool((got >= (ref * (1 - short)).to(t)).all()) and bool((got <= (ref * (1 + rounded)).to(t)).all())
