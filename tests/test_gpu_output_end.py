"""The output end's calls together: the example, a captured training step, two host
threads on one stream, calls after a launch that gave up."""
import importlib.util
import os
import threading

import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from dense_fp32_gemm_gb300 import layers

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("output_head", os.path.join(ROOT, "examples", "output_head.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def test_example_runs_and_serves():
    losses, norms, errors = example().run(tokens=200, vocabulary=777, width=136, steps=3)
    assert all(v == v and 0 < v < 100 for v in losses + norms)
    # 8 bits: two roundings, each off by at most half a step of 1/127 of a row's largest value (some four times its
    # root mean square); 4 bits: each off by at most a quarter of a value (of 3 and of 5 in 2 .. 6 units), some 10 %
    assert errors[0] < 0.03 and errors[1] < 0.25


def test_example_gradients():
    """Against autograd in 64 bits: G and the results in bf16, each off by 2^-9 of itself, the norm's output too."""
    e = example()
    t, v, h = 120, 500, 64
    x, r = rand(t, h).bfloat16(), rand(t, h, seed=1).bfloat16()
    target = torch.randint(0, v, (t,), generator=torch.Generator().manual_seed(2)).cuda()
    target[3] = -100
    gain, words = 1 + 0.1 * rand(h, seed=3), rand(v, h, seed=4, scale=0.2).bfloat16()
    leaves = [a.clone().requires_grad_() for a in (x, r, gain, words)]
    grads = torch.autograd.grad(e.loss_of(leaves[0], leaves[1], leaves[2], leaves[3], target), leaves)
    wide = [a.double().requires_grad_() for a in (x, r, gain, words)]
    s = wide[0] + wide[1]
    y = s / (s.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * wide[2]
    keep = target >= 0
    ref = torch.autograd.grad(torch.nn.functional.cross_entropy((y @ wide[3].mT)[keep], target[keep]), wide)
    for a, b in zip(grads, ref):
        # roundings of 2^-9 at h, at y, at G and at the result, and what y's and h's move in the probabilities (logits of
        # some 2, off by 2 * 2^-9 of them): below 8 * 2^-9 in the 2-norm
        assert float((a.double() - b).norm()) <= 8 * 2.0 ** -9 * float(b.norm())


def test_captured_training_step():
    """Norm, loss, both backward passes and the clipping in one graph, replayed on new inputs."""
    t, v, h = 64, 900, 128
    x, r = rand(t, h).bfloat16(), rand(t, h, seed=1).bfloat16()
    target = torch.randint(0, v, (t,), generator=torch.Generator().manual_seed(2)).cuda()
    gain = torch.ones(h, device="cuda", requires_grad=True)
    words = rand(v, h, seed=4, scale=0.1).bfloat16().requires_grad_()

    def step():
        y, _ = layers.rms_norm(x, gain, residual=r)
        loss = layers.linear_cross_entropy(y, words, target)
        grads = torch.autograd.grad(loss, [gain, words])
        return loss.detach(), B.clip_grad_norm(grads, 0.01), grads

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                           # sizes the stream's workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in (5, 6):
        x.copy_(rand(t, h, seed=seed))
        target.copy_(torch.randint(0, v, (t,), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(out[2], want[2]))


def test_layers_without_rows_or_columns():
    w = torch.ones(0, device="cuda", requires_grad=True)
    assert layers.rms_norm(torch.zeros(2, 3, 0, device="cuda"), w).shape == (2, 3, 0)
    x = torch.zeros(0, 4, 8, device="cuda", requires_grad=True)
    w = torch.ones(8, device="cuda", requires_grad=True)
    y, h = layers.rms_norm(x, w, residual=torch.zeros(0, 4, 8, device="cuda"))
    words = rand(5, 8).requires_grad_()
    loss = layers.linear_cross_entropy(y, words, torch.zeros(0, 4, dtype=torch.int64, device="cuda"))
    assert float(loss.detach()) == 0.0
    for g in torch.autograd.grad(loss, [x, w, words]):
        assert not bool(g.any())
    one = layers.rms_norm(rand(8), w)                      # a single row, without leading dimensions
    assert one.shape == (8,)


ROUNDS = 60


def test_two_host_threads_on_one_stream():
    """The launches of a call hand their data on in the stream's workspace, so they are queued together."""
    stream = torch.cuda.Stream()
    jobs, checks = [], []
    for i, dtype in enumerate((torch.bfloat16, torch.float32, torch.float16)):
        t, v, h = 100 + i, 700 + 100 * i, 101
        x, w = rand(t, h, seed=i).to(dtype), rand(v, h, seed=10 + i, scale=0.2).to(dtype)
        target = torch.randint(0, v, (t,), generator=torch.Generator().manual_seed(i)).cuda()
        d = rand(t, seed=20 + i)
        torch.cuda.synchronize()
        loss, lse = B.linear_cross_entropy(x, w, target)
        want = (loss, lse) + B.linear_cross_entropy_grad(x, w, target, lse, d)

        def job(x=x, w=w, target=target, d=d):
            loss, lse = B.linear_cross_entropy(x, w, target, stream=stream)
            return (loss, lse) + B.linear_cross_entropy_grad(x, w, target, lse, d, stream=stream)
        jobs.append(job)
        checks.append(want)
    y, g = rand(300, 512, seed=5).bfloat16(), rand(512, seed=6)
    _, hh, rstd = B.rms_norm(y, g)
    jobs.append(lambda: B.rms_norm_grad(y, hh, g, rstd, stream=stream))
    checks.append(B.rms_norm_grad(y, hh, g, rstd))
    torch.cuda.synchronize()
    start, got = threading.Barrier(len(jobs)), [None] * len(jobs)

    def loop(i):
        start.wait()
        got[i] = [jobs[i]() for _ in range(ROUNDS)]
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(jobs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for results, want in zip(got, checks):
        assert results is not None
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_after_a_launch_that_gave_up():
    """Cut tiles, before and after the status is polled: small integers, so that every order of sums is exact."""
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-1, 2, (80, 4000), generator=g).bfloat16().cuda()
    w = torch.randint(-1, 2, (500, 4000), generator=g).bfloat16().cuda()
    target = torch.randint(0, 500, (80,), generator=g).cuda()
    z = x.double() @ w.double().mT / 1.0
    lse = torch.logsumexp(z, dim=1)
    want = lse - z.gather(1, target[:, None])[:, 0]
    q, s = B.mx4_quantize(x[:3])
    qw, sw = B.mx4_quantize(w)
    stream = torch.cuda.current_stream().cuda_stream

    def calls():
        for rows in (slice(0, 80), slice(0, 5)):
            loss, _ = B.linear_cross_entropy(x[rows], w, target[rows])
            # exact logits; exponentials and their sum, 2e-6, and two roundings of some 200
            assert bool(((loss.double() - want[rows]).abs() <= 2e-6 + 2.0 ** -22 * lse[rows].abs()).all())
        assert torch.equal(B.mx4_gemm(q, s, qw, sw, out_dtype=torch.float32).double(), z[:3])

    calls()
    for _ in range(2):
        assert B.sgemm_diag_wait_timeout(1_000_000, stream) == 0           # 1 ms limit, runs out
        calls()
        assert B.sgemm_poll_device_status(stream) == (B.SGEMM_ERR_DEVICE_TIMEOUT, 1)
        calls()
        assert B.sgemm_poll_device_status(stream) == (0, 0)
