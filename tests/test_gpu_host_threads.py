"""Two host threads that call on one stream: the launches of a call (copies of
operands, then the product; the squares, then the scaling) are queued together,
since they hand their data on in the stream's workspace. ctypes releases the
interpreter's lock, so the threads do call at once."""
import threading

import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
ROUNDS = 150


def ints(shape, t, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(seed)).to(t).cuda()


def at_once(jobs):
    """Runs every job ROUNDS times, a thread each."""
    start = threading.Barrier(len(jobs))
    got = []

    def loop(job):
        start.wait()
        got.append([job() for _ in range(ROUNDS)])
    threads = [threading.Thread(target=loop, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == len(jobs) and all(st == 0 for g in got for st in g)


def grouped(seed, s, t, n, k):
    """A product whose operands are copied, into a result per round."""
    x, w = ints((40, k), t, seed), ints((2, n, k), t, seed + 1)
    off = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
    y = torch.zeros(ROUNDS, 40, n, device="cuda")
    code = {torch.bfloat16: B.SGEMM_TYPE_BF16, torch.float32: B.SGEMM_TYPE_F32}[t]
    turn = iter(range(1 << 30))

    def job():
        r = next(turn) % ROUNDS
        return B.sgemm_grouped(B.SGEMM_OP_T, code, B.SGEMM_TYPE_F32, 2, 40, n, k, 1.0, x.data_ptr(), k, w.data_ptr(),
                               k, n * k, off.data_ptr(), 0.0, y[r].data_ptr(), n, s)
    want = torch.cat([x[:15].double() @ w[0].double().mT, x[15:].double() @ w[1].double().mT])
    return job, lambda: bool((y.double() == want).all())


def x3(seed, s):
    a, b = ints((200, 1001), torch.float32, seed), ints((1001, 300), torch.float32, seed + 1)
    c = torch.zeros(ROUNDS, 200, 300, device="cuda")
    turn = iter(range(1 << 30))

    def job():
        r = next(turn) % ROUNDS
        return B.sgemm_3xtf32(200, 300, 1001, 1.0, a.data_ptr(), 1001, b.data_ptr(), 300, 0.0, c[r].data_ptr(), 300, s)
    want = a.double() @ b.double()
    return job, lambda: bool((c.double() == want).all())


def clip(value, s):
    g, out = torch.full((30000,), value, device="cuda"), torch.zeros(ROUNDS, 30000, device="cuda")
    norm = torch.zeros(ROUNDS, device="cuda")
    turn = iter(range(1 << 30))

    def job():
        r = next(turn) % ROUNDS
        return B.sgemm_grad_clip([g.data_ptr()], [out[r].data_ptr()], [30000], [B.SGEMM_TYPE_F32], 0.5 * value,
                                 norm[r].data_ptr(), s)

    def right():
        n = value * 30000 ** 0.5
        return bool(((norm - n).abs() < 1e-5 * n).all()) and bool(((out - 0.5 * value * value / n).abs() < 1e-5 * value).all())
    return job, right


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f32", "bf16"), ("x3", "bf16"), ("x3", "x3"), ("clip", "clip"),
                                   ("clip", "f32")], ids="-".join)
def test_calls_of_two_threads(kinds):
    stream = torch.cuda.Stream()
    s = stream.cuda_stream
    make = {"bf16": lambda i: grouped(10 * i, s, torch.bfloat16, 96 + i, 1001),
            "f32": lambda i: grouped(10 * i, s, torch.float32, 200, 333 + i),
            "x3": lambda i: x3(10 * i, s), "clip": lambda i: clip(1.0 + i, s)}
    made = [make[k](i) for i, k in enumerate(kinds)]
    torch.cuda.synchronize()
    for job, _ in made:          # the workspace has its size before the threads start
        assert job() == 0
    torch.cuda.synchronize()
    at_once([job for job, _ in made])
    assert all(right() for _, right in made)
    assert B.sgemm_poll_device_status(s) == (0, 0)


def test_growth_under_another_threads_calls():
    """One thread's operands grow call by call, so that the workspace moves."""
    stream = torch.cuda.Stream()
    s = stream.cuda_stream
    job, right = grouped(1, s, torch.bfloat16, 96, 1001)
    sizes = iter(range(1 << 30))
    x, w = torch.ones(2, 4000 * 1001 + 1, device="cuda"), torch.ones(4000 * 1001, device="cuda")
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    y = torch.zeros(ROUNDS, 2, 4000, device="cuda")

    def growing():
        r = next(sizes) % ROUNDS
        n = 100 + 26 * r
        return B.sgemm_grouped(B.SGEMM_OP_T, B.SGEMM_TYPE_F32, B.SGEMM_TYPE_F32, 1, 2, n, 1001, 1.0, x.data_ptr(), 1001,
                               w.data_ptr(), 1001, 0, off.data_ptr(), 0.0, y[r].data_ptr(), 4000, s)
    torch.cuda.synchronize()
    at_once([job, growing])
    assert right()
    for r in range(ROUNDS):
        n = 100 + 26 * r
        assert bool((y[r, :, :n] == 1001).all()) and not bool(y[r, :, n:].any())
