"""The two ways of an 8-bit product: operands converted tile by tile, or widened
to F16 first. By the measured times of both, and forced by the tile's width."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ints(shape, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.randint(-128, 128, (shape[0], shape[1] + pad), generator=g, dtype=torch.int8, device="cuda")
    return store[:, pad:]


def check(m, n, k, pad=0):
    a, b = ints((m, k), m, pad), ints((n, k), n + k, 2 * pad)
    sa, sb = torch.full((m,), 0.25, device="cuda"), torch.full((n,), 2.0, device="cuda")
    got = B.i8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    assert torch.equal(got.double(), ((a.double() @ b.double().mT) * 0.5).float().double())
    assert B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream) == (0, 0)
    return B.sgemm_last_config()


# measured: which side is faster, by 10 % and more
@pytest.mark.parametrize("m,n,k,wide", [(1, 4096, 4096, False), (512, 4096, 4096, False), (600, 512, 512, False),
                                        (2048, 1024, 4096, False), (2048, 512, 512, False), (256, 14336, 4096, False),
                                        (1024, 4096, 4096, True), (2048, 4096, 1024, True), (1024, 14336, 4096, True),
                                        (384, 8191, 1000, True), (256, 8191, 1000, False)])
def test_the_faster_form(m, n, k, wide):
    assert ("256x256x64" in check(m, n, k)) == wide


@pytest.mark.parametrize("form", [(256, 1), (256, 2)], ids=str)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (70, 130, 65), (512, 130, 1000), (513, 264, 65), (1500, 777, 2049), (700, 1030, 16)])
@pytest.mark.parametrize("pad", [0, 3])
def test_widened_by_request(form, m, n, k, pad):
    assert B.sgemm_grouped_set_tile(*form) == 0
    try:
        assert f"{128 * form[1]}x256x64" in check(m, n, k, pad)
    finally:
        assert B.sgemm_grouped_set_tile(0) == 0


@pytest.mark.parametrize("form", [(16, 1), (128, 1)], ids=str)
def test_tile_by_tile_by_request(form):
    assert B.sgemm_grouped_set_tile(*form) == 0
    try:
        assert f"128x{form[0]}x" in check(1100, 2100, 520)
    finally:
        assert B.sgemm_grouped_set_tile(0) == 0
