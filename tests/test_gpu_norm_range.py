"""The norm of long rows of the largest values: squares that FP32 does not hold are
summed once more, scaled down, and the scaled sum has to stay in range, too.

Tolerances: as in the tests of the norm (36 * 2^-24 for 1 / rms, 40 for y, 38 for the
scale, at most 64 additions one after another). 1 / rms of values above 8e37 lies
below FP32's normal numbers and is stored in steps of 2^-149, of values up to 2^128
within 2^-150 / 2^-128 = 2^-22 of itself: 4 * 2^-24 more."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rounding(want, t):
    f = torch.finfo(t)
    return torch.maximum(want.abs() * f.eps / 2, torch.full_like(want, f.smallest_normal * f.eps / 2))


# (the last two rows do not start on 16 bytes: by shifted pieces, by single elements)
@pytest.mark.parametrize("n", [128, 600, 8192, 16384, 65536, 16383, 65535])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
def test_the_largest_values(t, n):
    most = torch.finfo(t).max
    g = torch.Generator(device="cuda").manual_seed(n)
    sign = torch.where(torch.rand(5, n, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    f = sign.double() * most
    f[1] *= 0.75
    f[2] *= torch.rand(n, generator=g, device="cuda").double()
    f[3] *= 2.0 ** -30
    f[4, 1:] = 0                                 # one value alone
    x = f.to(t)
    f = x.double()
    w = (1 + 0.25 * torch.randn(n, generator=g, device="cuda")).clamp(0.5, 1.0)
    y, _, rstd = B.rms_norm(x, w)
    ref = 1 / (f.square().mean(dim=1) + 1e-6).sqrt()
    assert bool(((rstd.double() - ref).abs() <= ref * 40 * U).all()), (rstd, ref)
    want = f * ref[:, None] * w.double()
    assert bool(((y.double() - want).abs() <= rounding(want, t) + want.abs() * 44 * U).all())
    q, scale, _ = B.rms_norm_i8(x, w)
    step = ((f * w.double()).float().double().abs().amax(dim=1) / 127).float().double()
    assert torch.equal(q.double(), ((f * w.double()).float().double() / step[:, None]).float().double().round().clamp(-127, 127))
    assert bool(((scale.double() - step * ref).abs() <= step * ref * 42 * U).all()), (scale, step * ref)
