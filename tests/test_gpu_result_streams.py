"""A call on a stream of its own, without a result tensor: the result is that
stream's own allocation. One of the current stream's would be a block that
work queued there still writes (and would go back to that stream while the
kernel has yet to write it)."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def ints(shape, t, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(seed)).to(t).cuda()


def pending(shapes):
    """Leaves freed blocks of these shapes and types behind, which the current
    stream writes only some 50 ms from now."""
    blocks = [torch.empty(shape, dtype=t, device="cuda") for shape, t in shapes]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for b in blocks:
        b.fill_(7)


def cases():
    x, w, dy = ints((2000, 64), BF16, 1), ints((2, 96, 64), BF16, 2), ints((2000, 96), BF16, 3)
    off = torch.tensor([0, 700, 2000], dtype=torch.int32, device="cuda")
    q, qw = ints((2000, 64), torch.int8, 4), ints((96, 64), torch.int8, 5)
    one, onew = torch.ones(2000, device="cuda"), torch.ones(96, device="cuda")
    x[:, 0] = 127                # so that the scales are 1
    grads = [torch.full((3000,), 3.0, device="cuda"), torch.full((3000,), 4.0, device="cuda")]
    y = torch.cat([x[:700].float() @ w[0].float().mT, x[700:].float() @ w[1].float().mT])
    dw = torch.stack([dy[:700].float().mT @ x[:700].float(), dy[700:].float().mT @ x[700:].float()])
    f32 = torch.float32
    return {
        "rows": ([((2000, 96), f32)], lambda s: [B.grouped_gemm(x, w, off, out_dtype=f32, stream=s)], [y]),
        "wgrad": ([((2, 96, 64), f32)], lambda s: [B.grouped_wgrad(dy, x, off, out_dtype=f32, stream=s)], [dw]),
        "quantize": ([((2000, 64), torch.int8), ((2000,), f32)], lambda s: list(B.i8_quantize(x, stream=s)),
                     [x.to(torch.int8), one]),
        "i8": ([((2000, 96), f32)], lambda s: [B.i8_gemm(q, one, qw, onew, out_dtype=f32, stream=s)],
               [q.float() @ qw.float().mT]),
        "clip": ([((), f32)], lambda s: [B.clip_grad_norm(grads, 1e9, stream=s)],
                 [torch.tensor(75000.0, device="cuda").sqrt()]),
    }


@pytest.mark.parametrize("name", ["rows", "wgrad", "quantize", "i8", "clip"])
def test_results_belong_to_the_given_stream(name):
    shapes, call, want = cases()[name]
    s = torch.cuda.Stream()
    call(s)                      # the stream's workspace
    torch.cuda.synchronize()
    pending(shapes)
    got = call(s)
    s.synchronize()
    kept = [t.clone() for t in got]
    torch.cuda.synchronize()
    for g, k, w in zip(got, kept, want):
        assert torch.equal(g, w) and torch.equal(k, w)
    # released while the stream has yet to write them, they are not handed out
    # to the current stream
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    ptrs = {t.data_ptr() for t in call(s)}
    del got, kept
    again = [torch.zeros(shape, dtype=t, device="cuda") for shape, t in shapes]
    torch.cuda.synchronize()
    assert not ptrs & {t.data_ptr() for t in again}
    assert not any(bool(t.any()) for t in again)


def test_current_stream_and_device_come_back():
    shapes, call, want = cases()["rows"]
    before = torch.cuda.current_stream()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(None)
        assert torch.cuda.current_stream() == s
    call(s)
    assert torch.cuda.current_stream() == before
    with pytest.raises(B.SgemmError):
        B.grouped_gemm(torch.zeros(4, 8, device="cuda"), torch.zeros(1025, 8, 8, device="cuda"),
                       torch.zeros(1026, dtype=torch.int32, device="cuda"), stream=s)
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])


def test_default_stream_by_name():
    shapes, call, want = cases()["rows"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
