"""A captured graph keeps the workspace block it was captured with: a later,
larger call on the stream gets another block, and replays stay right. (Freed,
the block would be read and written by the replays.)"""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ints(shape, t, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(seed)).to(t).cuda()


def grow(s, floats):
    """Calls on `s` whose operands have to be copied: the workspace holds the copies."""
    k = 1001
    n = floats // k
    x, w = torch.ones(8, k, device="cuda"), torch.ones(1, n, k, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    y = torch.empty(8, n, device="cuda")
    torch.cuda.synchronize()
    B.grouped_gemm(x, w, off, Y=y, stream=s)
    s.synchronize()
    assert bool((y == k).all())


def capture(s, call):
    call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    return graph


def test_replays_after_growth():
    s = torch.cuda.Stream()
    # an unaligned operand (copied into the workspace) and tiles cut along k
    x, w = ints((20, 2049), torch.bfloat16, 1), ints((2, 256, 2049), torch.bfloat16, 2)
    off = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    y = torch.zeros(20, 256, device="cuda")
    a, b = ints((256, 9000), torch.float32, 3), ints((9000, 512), torch.float32, 4)
    c = torch.zeros(256, 512, device="cuda")
    g = [ints((5000,), torch.float32, 5)]
    out = [torch.zeros(5000, device="cuda")]
    norm = {}

    def products():
        B.grouped_gemm(x, w, off, Y=y, stream=s)
        for call in (B.sgemm, B.sgemm_3xtf32):
            assert call(256, 512, 9000, 1.0, a.data_ptr(), 9000, b.data_ptr(), 512, 1.0 if call is B.sgemm_3xtf32 else 0.0,
                        c.data_ptr(), 512, s.cuda_stream) == 0
        norm["t"] = B.clip_grad_norm(g, 1e9, out=out, stream=s)

    torch.cuda.synchronize()
    graphs = [capture(s, products)]
    for floats in (1 << 24, 1 << 26):
        grow(s, floats)
        graphs.append(capture(s, products))     # a block for each
    fill = torch.full((1 << 26,), float("nan"), device="cuda")   # what a freed block's memory could hold
    for r, graph in enumerate(graphs * 2):
        x.copy_(ints((20, 2049), torch.bfloat16, 10 + r))
        a.copy_(ints((256, 9000), torch.float32, 30 + r))
        g[0].copy_(ints((5000,), torch.float32, 50 + r))
        for t in (y, c, out[0]):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.cat([x[:7].double() @ w[0].double().mT, x[7:].double() @ w[1].double().mT])
        assert torch.equal(y.double(), want)
        assert torch.equal(c.double(), 2 * (a.double() @ b.double()))
        assert torch.equal(out[0], g[0])
    assert bool(fill.isnan().all())
    assert B.sgemm_poll_device_status(s.cuda_stream) == (0, 0)


def test_status_of_a_graph_with_a_retired_block():
    s = torch.cuda.Stream()

    def wait():
        assert B.sgemm_diag_wait_timeout(1_000_000, s.cuda_stream) == 0   # 1 ms limit

    graph = capture(s, wait)
    assert B.sgemm_poll_device_status(s.cuda_stream)[0] == B.SGEMM_ERR_DEVICE_TIMEOUT
    grow(s, 1 << 22)
    graph.replay()
    torch.cuda.synchronize()
    assert B.sgemm_poll_device_status(s.cuda_stream) == (B.SGEMM_ERR_DEVICE_TIMEOUT, 1)
    assert B.sgemm_poll_device_status(s.cuda_stream) == (0, 0)
