"""Host threads that call the norm at once, each on a stream of its own, with rows
that do not start on 16 bytes: a call's kernel takes the weights into shared memory, as
much as its rows need, and another thread's call of shorter rows must not lower what
the kernel may take. ctypes releases the interpreter's lock, so the threads do call at
once."""
import threading

import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
ROUNDS = 4000


def norm(n, form, seed):
    """A forward call of two rows of n values (n odd) on its own stream: the job, whether its output is right, and
    what it uses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-3, 4, (2, n), generator=g, device="cuda").bfloat16()
    w = torch.ones(n, device="cuda")
    stream = torch.cuda.Stream()
    s = stream.cuda_stream
    out = torch.zeros(2, n, dtype=torch.bfloat16 if form == "y" else torch.int8, device="cuda")
    rows = torch.zeros(2, device="cuda")
    args = (2, n, B.SGEMM_TYPE_BF16, x.data_ptr(), n, None, n, w.data_ptr(), B.SGEMM_TYPE_F32, 1e-6, None, n,
            out.data_ptr(), n, rows.data_ptr(), s)

    def job():
        return B.sgemm_rms_norm(*args) if form == "y" else B.sgemm_rms_norm_i8(*args)

    def right():
        f = x.double()
        if form != "y":
            u = x.float() / (x.float().abs().amax(dim=1) / 127)[:, None]
            return torch.equal(out.float(), u.round().clamp(-127, 127))
        want = f / (f.square().mean(dim=1, keepdim=True) + 1e-6).sqrt()
        # half a step of BF16 and FP32 sums
        return bool(((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18)).all())
    return job, right, (stream, w, rows)           # (what the calls use lives as long as the job)


@pytest.mark.parametrize("form", ["y", "i8"])
def test_rows_of_different_lengths_at_once(form):
    made = [norm(n, form, i) for i, n in enumerate((20001, 13001, 9001, 23001))]    # 36 to 92 KB of weights
    torch.cuda.synchronize()
    for job, _, _ in made:
        assert job() == 0
    torch.cuda.synchronize()
    start, got = threading.Barrier(len(made)), []

    def loop(job):
        start.wait()
        got.append({job() for _ in range(ROUNDS)})
    threads = [threading.Thread(target=loop, args=(job,)) for job, _, _ in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert got == [{0}] * len(made)
    assert all(right() for _, right, _ in made)
