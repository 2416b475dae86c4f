"""Sizes at the ends of the 32-bit range: places in a row and row numbers that
pass 2^31 when they are stepped on."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def pattern(n):
    """Values of a period that no block or grid size shares, from +-3 to +-125."""
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 1 << 28):
        b = min(n, a + (1 << 28))
        i = torch.arange(a, b, device="cuda")
        x[a:b] = ((i % 61 + 1) * 2 + 1).to(torch.bfloat16) * torch.where(i % 7 < 3, -1.0, 1.0).to(torch.bfloat16)
    return x


def chunks(n, step=1 << 28):
    return [slice(a, min(n, a + step)) for a in range(0, n, step)]


def test_quantize_most_rows():
    """2^31 - 1 rows of one value: each is +-127 of its own scale."""
    x = pattern(MOST)
    q, s = torch.zeros(MOST, 1, dtype=torch.int8, device="cuda"), torch.zeros(MOST, device="cuda")
    B.i8_quantize(x.view(MOST, 1), Q=q, scale=s)
    most = torch.tensor(127.0, device="cuda")   # (by a Python number torch multiplies by its reciprocal)
    for c in chunks(MOST):
        assert torch.equal(q[c, 0], (torch.sign(x[c]) * 127).to(torch.int8))
        assert torch.equal(s[c], x[c].float().abs() / most)


def test_quantize_longest_row():
    x = pattern(MOST)
    x[MOST - 1] = 127.0                  # the scale is 1
    q, s = torch.zeros(1, MOST, dtype=torch.int8, device="cuda"), torch.zeros(1, device="cuda")
    B.i8_quantize(x.view(1, MOST), Q=q, scale=s)
    assert float(s) == 1.0
    for c in chunks(MOST):
        assert torch.equal(q[0, c], x[c].to(torch.int8))


@pytest.mark.parametrize("k", [2 ** 29 + 5, 2 ** 29 - 3])
def test_copied_rows_of_two_gigabytes(k):
    """FP32 rows that have to be copied, of more bytes than 32 bits count (and of just fewer)."""
    x, w = torch.zeros(2, k, device="cuda"), torch.zeros(1, 1, k, device="cuda")
    at = torch.tensor([0, 1, 15, 16, 12345, 2 ** 27 + 3, 2 ** 28 - 1, 2 ** 28, 2 ** 29 - 13, k - 6, k - 2, k - 1], device="cuda")
    w[0, 0, at] = torch.arange(1, len(at) + 1, device="cuda").float()
    x[0, at] = 1.0
    x[1, at] = torch.arange(len(at), device="cuda").float()
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    y = B.grouped_gemm(x, w, off)
    assert "p=copied q=copied" in B.sgemm_last_config()
    n = len(at)
    assert y.flatten().tolist() == [n * (n + 1) / 2, sum(i * (i + 1) for i in range(n))]
    assert B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream) == (0, 0)
    B.sgemm_shutdown()                   # (a workspace of 6 GB)
