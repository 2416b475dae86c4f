"""What lies between the rows of matrices that the 4-bit calls write stays as it is, where
rows start on 16 bytes and end inside 16, too. Values are small integers that 4 bits
hold, so every product is exact in any order."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def ints(m, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, (m, k), generator=g, device="cuda").float()


def padded(m, n, t, unit):
    """A matrix of m x n whose rows start at multiples of `unit` elements, at least one element apart; its store."""
    pitch = (n + unit) // unit * unit
    store = torch.full((m * pitch + unit,), 77, dtype=t, device="cuda")
    return store, store[:m * pitch].view(m, pitch)


@pytest.mark.parametrize("tile", [(0, 1), (128, 1), (256, 1), (256, 2)])
@pytest.mark.parametrize("m,n,k", [(365, 46, 1064), (764, 13, 40), (300, 1, 64), (129, 259, 8), (700, 1003, 1000),
                                   (257, 33, 9000), (300, 1028, 520), (20, 333, 700), (1, 4099, 4096)])
@pytest.mark.parametrize("t", TYPES)
def test_product(t, m, n, k, tile):
    a, b = ints(m, k, 1), ints(n, k, 2)
    want = (a.double() @ b.double().mT).to(t)
    operands = B.mx4_quantize(a) + B.mx4_quantize(b)
    for unit in (16 // t.itemsize, 64):
        store, rows = padded(m, n, t, unit)
        try:
            assert B.sgemm_grouped_set_tile(*tile) == 0
            B.mx4_gemm(*operands, C=rows[:, :n])
        finally:
            B.sgemm_grouped_set_tile(0)
        assert torch.equal(rows[:, :n], want)
        assert bool((rows[:, n:] == 77).all()) and bool((store[rows.numel():] == 77).all())


@pytest.mark.parametrize("m,k", [(300, 1), (129, 13), (70, 46), (9, 1003), (200, 4100)])
@pytest.mark.parametrize("t", TYPES)
def test_rounding_and_back(t, m, k):
    x = ints(m, k, 3).to(t)
    q0, s0 = B.mx4_quantize(x)
    codes = q0.shape[1]
    store, rows = padded(m, codes, torch.uint8, 16)
    scales = torch.full((s0.numel() + 16,), 77, dtype=torch.uint8, device="cuda")
    B.mx4_quantize(x, Q=rows[:, :codes], scale=scales[:-16])
    assert torch.equal(rows[:, :codes], q0) and torch.equal(scales[:-16], s0)
    assert bool((rows[:, codes:] == 77).all()) and bool((store[rows.numel():] == 77).all())
    assert bool((scales[-16:] == 77).all())
    for unit in (16 // t.itemsize, 64):
        store, rows = padded(m, k, t, unit)
        B.mx4_dequantize(q0, s0, k, X=rows[:, :k])
        assert torch.equal(rows[:, :k], x)
        assert bool((rows[:, k:] == 77).all()) and bool((store[rows.numel():] == 77).all())
