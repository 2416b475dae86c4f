"""Calls after a launch that gave up on a wait, before and after its status is
polled. Such a launch can leave flags and arrival counters behind (the
diagnostic leaves both): the next calls must not take them for their own."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ints(shape, t, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(seed)).to(t).cuda()


@pytest.mark.parametrize("form", [None, (16, 1), (64, 1), (256, 1), (256, 2)], ids=str)
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_cut_tiles(form, t):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[t]
    x, w = ints((300, 4096), t, 1), ints((3, 256, 4096), t, 2)
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    want = torch.cat([x[:100].double() @ w[0].double().mT, x[100:].double() @ w[2].double().mT])
    a, b = ints((4096, 130), t, 3), ints((4096, 140), t, 4)
    offb = torch.tensor([0, 3000, 4096], dtype=torch.int32, device="cuda")
    wantb = torch.stack([a[:3000].double().mT @ b[:3000].double(), a[3000:].double().mT @ b[3000:].double()])
    c, d = ints((256, 9000), torch.float32, 5), ints((9000, 512), torch.float32, 6)
    wantc = c.double() @ d.double()
    s = torch.cuda.current_stream().cuda_stream

    def calls():
        y = B.grouped_gemm(x, w, off, out_dtype=torch.float32)
        g = B.grouped_wgrad(a, b, offb, out_dtype=torch.float32)
        assert torch.equal(y.double(), want) and torch.equal(g.double(), wantb)
        for call in (B.sgemm, B.sgemm_3xtf32):
            e = torch.empty(256, 512, device="cuda")
            assert call(256, 512, 9000, 1.0, c.data_ptr(), 9000, d.data_ptr(), 512, 0.0, e.data_ptr(), 512, s) == 0
            assert torch.equal(e.double(), wantc)

    if form is not None:
        assert B.sgemm_grouped_set_tile(*form) == 0
    try:
        calls()
        for _ in range(2):
            assert B.sgemm_diag_wait_timeout(1_000_000, s) == 0       # 1 ms limit, runs out
            calls()
            calls()
            assert B.sgemm_poll_device_status(s) == (B.SGEMM_ERR_DEVICE_TIMEOUT, 1)
            calls()
            assert B.sgemm_poll_device_status(s) == (0, 0)
    finally:
        assert B.sgemm_grouped_set_tile(0) == 0


def test_replay_of_a_graph():
    x, w = ints((20, 4096), torch.bfloat16, 1), ints((1, 256, 4096), torch.bfloat16, 2)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    y = torch.zeros(20, 256, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    B.grouped_gemm(x, w, off, Y=y, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.grouped_gemm(x, w, off, Y=y)
    assert B.sgemm_diag_wait_timeout(1_000_000, s.cuda_stream) == 0
    for _ in range(2):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.double(), x.double() @ w[0].double().mT)
    assert B.sgemm_poll_device_status(s.cuda_stream)[0] == B.SGEMM_ERR_DEVICE_TIMEOUT
