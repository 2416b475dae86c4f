"""sgemm_i8_quantize and sgemm_i8 against integer and 64-bit references.

The integer sum is exact, so with scales that are powers of two an FP32 result
is the integer rounded once; with other scales two further FP32 products are
rounded (3 * 2^-24 relative), then the output type (2^-8, 2^-11).
"""
import numpy as np
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def ints(shape, seed, ld=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    ld = ld or shape[1]
    store = torch.full((offset + shape[0] * ld + 64,), 101, dtype=torch.int8, device="cuda")
    view = store[offset: offset + shape[0] * ld].view(shape[0], ld)[:, :shape[1]]
    view.copy_(v)
    return v, view


def exact_sum(a, b):
    return (a.cuda().double() @ b.cuda().double().mT)   # below 2^53: exact


@pytest.mark.parametrize("m", [1, 2, 31, 33, 65, 130, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 16), (127, 65), (129, 200), (264, 1040)])
def test_exact_sums(m, n, k):
    a, da = ints((m, k), m)
    b, db = ints((n, k), n + k)
    sa, sb = torch.full((m,), 0.5, device="cuda"), torch.full((n,), 4.0, device="cuda")
    got = B.i8_gemm(da, sa, db, sb, out_dtype=torch.float32)
    assert B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream)[0] == 0
    assert torch.equal(got, (exact_sum(a, b) * 2.0).float())


@pytest.mark.parametrize("m", [1, 70])
@pytest.mark.parametrize("value", [-128, 127])
def test_extreme_values_stay_exact(m, value):
    for k in (1025, 20000, B.SGEMM_I8_MAX_K):
        a = torch.full((m, k), value, dtype=torch.int8, device="cuda")
        b = torch.full((130, k), -128, dtype=torch.int8, device="cuda")
        one_m, one_n = torch.ones(m, device="cuda"), torch.ones(130, device="cuda")
        got = B.i8_gemm(a, one_m, b, one_n, out_dtype=torch.float32)
        want = torch.tensor(float(np.float32(value * -128 * k)), device="cuda")
        assert bool((got == want).all())


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k,pads,offs", [(5, 100, 300, (0, 0, 0), (0, 0)), (140, 515, 777, (3, 9, 5), (1, 7)),
                                             (300, 264, 4096, (16, 32, 8), (16, 16))])
def test_scales_strides_types(out, m, n, k, pads, offs):
    a, da = ints((m, k), 1, k + pads[0], offs[0])
    b, db = ints((n, k), 2, k + pads[1], offs[1])
    g = torch.Generator().manual_seed(3)
    sa = (torch.rand((m,), generator=g) * 1e-3).cuda()
    sb = (torch.rand((n,), generator=g) * 1e-2).cuda()
    store = torch.full((m, n + pads[2]), float("nan"), dtype=TYPES[out], device="cuda")
    C = store[:, :n]
    B.i8_gemm(da, sa, db, sb, C=C)
    ref = exact_sum(a, b) * sa.double()[:, None] * sb.double()
    tol = (ROUND[TYPES[out]] + 3 * 2.0 ** -24) * ref.abs() + (2.0 ** -24 if out == "f16" else 1e-38)
    assert bool(((C.double() - ref).abs() <= tol).all())
    assert bool(store[:, n:].isnan().all())


def reference_quantize(x):
    """The definition in NumPy: FP32 quotients (correctly rounded), ties to even."""
    x = x.numpy().astype(np.float32)
    scale = (np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)) / np.float32(127)
    safe = np.where(scale > 0, scale, np.float32(1))
    q = np.clip(np.rint(x / safe[:, None]), -127, 127)
    return np.where(scale[:, None] > 0, q, 0).astype(np.int8), scale.astype(np.float32)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (17, 255), (40, 4096), (500, 1000), (2, 70001), (700, 1000), (900, 4096),
                                 (650, 4100), (1300, 33)])
def test_quantize(t, m, k):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn((m, k), generator=g)
    x[:, :: 7] *= 30.0
    if k >= 128:
        # half-way cases: amax 127 makes the scale 1 and x.5 a tie
        x[0] = (torch.randint(-126, 126, (k,), generator=g) + 0.5).clamp(-127, 127)
        x[0, 5] = 127.0
    x[m // 2] *= 0.0 if m > 2 else 1.0
    x = x.to(TYPES[t])
    want_q, want_s = reference_quantize(x.float())
    q, s = B.i8_quantize(x.cuda())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_strides_and_padding():
    x = torch.randn((9, 50)).bfloat16()
    store = torch.full((9, 61), float("nan"), dtype=torch.bfloat16, device="cuda")
    store[:, 3:53] = x.cuda()
    Q = torch.full((9, 77), 99, dtype=torch.int8, device="cuda")
    q, s = B.i8_quantize(store[:, 3:53], Q=Q[:, 5:55])
    want_q, want_s = reference_quantize(x.float())
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    assert bool((Q[:, :5] == 99).all()) and bool((Q[:, 55:] == 99).all())


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantize_tiny_huge_and_non_finite_rows(t):
    big = {"f32": 3.4e38, "bf16": 3.3e38, "f16": 65504.0}[t]
    tiny = {"f32": 1e-45, "bf16": 1e-40, "f16": 6e-8}[t]
    x = torch.zeros((5, 64), dtype=TYPES[t])
    x[0, 3], x[0, 4] = big, -big
    x[1, :] = tiny
    x[2, 7], x[2, 8] = float("inf"), 1.0
    x[3, 9], x[3, 10] = float("nan"), 2.0
    q, s = B.i8_quantize(x.cuda())
    want_q, want_s = reference_quantize(x[:2].float())
    assert np.array_equal(q[:2].cpu().numpy(), want_q) and np.array_equal(s[:2].cpu().numpy(), want_s)
    assert float(s[2]) == float("inf") and bool(s[3].isnan()) and float(s[4]) == 0.0
    assert bool((q[2:] == 0).all())
    w = torch.ones((8, 64), dtype=torch.int8, device="cuda")
    y = B.i8_gemm(q, s, w, torch.ones(8, device="cuda"), out_dtype=torch.float32)
    assert bool(y[2:4].isnan().all()) and bool((y[4] == 0).all())


def test_quantised_linear_layer():
    """Both calls as a layer runs them, on a stream of their own and in a graph."""
    x = torch.randn((70, 512)).bfloat16().cuda()
    w, dw = ints((200, 512), 4)
    sw = torch.rand(200).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q, sx = B.i8_quantize(x)
        y = B.i8_gemm(q, sx, dw, sw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            B.i8_quantize(x, Q=q, scale=sx)
            B.i8_gemm(q, sx, dw, sw, C=y)
        x.copy_(torch.randn((70, 512)).bfloat16())
        graph.replay()
    s.synchronize()
    want_q, want_s = reference_quantize(x.cpu().float())
    ref = exact_sum(torch.from_numpy(want_q), w) * torch.from_numpy(want_s).cuda().double()[:, None] * sw.double()
    assert bool(((y.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -22) * ref.abs()).all())


@pytest.mark.parametrize("m,n,k", [(512, 130, 1000), (513, 264, 65), (1500, 777, 2049), (700, 1030, 16)])
@pytest.mark.parametrize("pads", [0, 3])
def test_many_rows(m, n, k, pads):
    """The widened path: whole and cut tiles, odd edges, unaligned rows."""
    a, da = ints((m, k), m, k + pads, pads)
    b, db = ints((n, k), n + k, k + pads, 2 * pads)
    sa, sb = torch.full((m,), 0.25, device="cuda"), torch.full((n,), 2.0, device="cuda")
    got = B.i8_gemm(da, sa, db, sb, out_dtype=torch.float32)
    assert B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream)[0] == 0
    assert torch.equal(got, (exact_sum(a, b) * 0.5).float())


@pytest.mark.parametrize("form", [(16, 1), (32, 1), (64, 1), (128, 1), (256, 1), (256, 2)], ids=str)
@pytest.mark.parametrize("m", [70, 600])
def test_every_tile(form, m):
    a, da = ints((m, 2100), 1)
    b, db = ints((300, 2100), 2)
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(300, device="cuda")
    assert B.sgemm_grouped_set_tile(*form) == 0
    try:
        got = B.i8_gemm(da, one_m, db, one_n, out_dtype=torch.float32)
    finally:
        assert B.sgemm_grouped_set_tile(0) == 0
    assert torch.equal(got, exact_sum(a, b).float())


@pytest.mark.parametrize("m", [40, 600])
@pytest.mark.parametrize("k", [37, 1100])
def test_every_byte_alignment(m, k):
    """Start addresses and pitches of every remainder by 16, one row a piece longer than the last."""
    sa, sb = torch.ones(m, device="cuda"), torch.ones(130, device="cuda")
    for r in range(16):
        a, da = ints((m, k), r, k + r, 16 - r)
        b, db = ints((130, k), 100 + r, k + (5 * r) % 16, r)
        assert torch.equal(B.i8_gemm(da, sa, db, sb, out_dtype=torch.float32), exact_sum(a, b).float())
