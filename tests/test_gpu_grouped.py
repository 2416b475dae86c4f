"""sgemm_grouped and sgemm_grouped_wgrad against products in 64 bits.

Tolerance, per element: u_out * |ref| for the one rounding to the output type
(2^-8, 2^-11, 2^-24 for bf16, f16, f32), plus 2 * n * 2^-23 * sum |x||w| for the
sum, n being the number of truncating additions into one accumulator and of
the rounded ones behind it: K/16 for 16-bit results, 16 + K/256 for 32-bit
results of 16-bit operands, 24 + K/64 for FP32 operands (plus 4 for the
products kept). Small integers have to come out exactly.
"""
import numpy as np
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def additions(k, t, out):
    if t == torch.float32:
        return 28 + k / 64
    return 16 + k / 256 + 2 if out == torch.float32 else k / 16 + 2


def values(shape, t, seed, ints=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-3, 4, shape, generator=g).float() if ints else torch.randn(shape, generator=g)
    return v.to(t)


def padded(host, ld, offset=0):
    """A device copy with row pitch `ld` (last dimension) and `offset` elements
    before it, NaN everywhere else."""
    lead, rows, cols = (1,) * (3 - host.dim()) + tuple(host.shape)
    store = torch.full((offset + lead * rows * ld + 64,), float("nan"), dtype=host.dtype, device="cuda")
    view = store[offset: offset + lead * rows * ld].view(lead, rows, ld)[:, :, :cols]
    view.copy_(host.view(lead, rows, cols))
    return view if host.dim() == 3 else view[0]


def assert_close(got, ref, mag, n):
    u = ROUND[got.dtype]
    tol = u * ref.abs() + 2 * n * 2.0 ** -23 * mag + 2.0 ** -24 * (got.dtype == torch.float16) + 1e-37
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off; worst "
                                 f"{float(((got.double() - ref).abs() / tol).max()):.3g} of the tolerance")


def bounds_of(counts, start=0):
    return [start] + (start + np.cumsum(counts)).tolist()


def run_rows(op, t, out, counts, n, k, ints=False, alpha=1.0, beta=0.0, pads=(0, 0, 0), offs=(0, 0, 0),
             lead=0, tail=0, seed=0):
    e, rows = len(counts), lead + sum(counts) + tail
    x = values((rows, k), t, seed, ints)
    w = values((e, n, k) if op == "T" else (e, k, n), t, seed + 1, ints)
    y0 = values((rows, n), out, seed + 2, ints)
    bounds = bounds_of(counts, lead)
    X, W = padded(x, k + pads[0], offs[0]), padded(w, w.size(2) + pads[1], offs[1])
    Y = padded(y0, n + pads[2], offs[2])
    if beta == 0.0:
        Y.fill_(float("nan"))
    before = Y.clone()
    store = Y._base if Y._base is not None else Y
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    B.grouped_gemm(X, W, offsets, Y=Y, op=op, alpha=alpha, beta=beta)
    st, detail = B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream)
    assert st == 0, detail
    xd, wd, yd = x.cuda().double(), w.cuda().double(), y0.cuda().double()
    for i in range(e):
        a, b = bounds[i], bounds[i + 1]
        if a == b:
            continue
        we = wd[i].mT if op == "T" else wd[i]
        ref = alpha * (xd[a:b] @ we) + (beta * yd[a:b] if beta else 0.0)
        if ints:
            assert torch.equal(Y[a:b], ref.to(out)), f"group {i}"
        else:
            mag = abs(alpha) * (xd[a:b].abs() @ we.abs()) + abs(beta) * yd[a:b].abs()
            assert_close(Y[a:b], ref, mag, additions(k, t, out))
    # rows outside the groups, and the padding, are not touched
    for sl in (slice(0, bounds[0]), slice(bounds[-1], rows)):
        assert torch.equal(Y[sl].nan_to_num(7.5), before[sl].nan_to_num(7.5))
    if pads[2]:
        whole = store.flatten()[offs[2]: offs[2] + rows * (n + pads[2])].view(rows, n + pads[2])
        assert bool(whole[:, n:].isnan().all())
    return Y


def run_wgrad(t, out, counts, m, n, ints=False, alpha=1.0, beta=0.0, pads=(0, 0, 0), offs=(0, 0, 0),
              lead=0, tail=0, seed=0):
    e, rows = len(counts), lead + sum(counts) + tail
    a = values((rows, m), t, seed, ints)
    b = values((rows, n), t, seed + 1, ints)
    bounds = bounds_of(counts, lead)
    # rows of no group hold NaN: they must not reach any sum
    for v in (a, b):
        v[:lead] = float("nan")
        v[rows - tail:] = float("nan")
    c0 = values((e, m, n), out, seed + 2, ints)
    A, Bm, C = padded(a, m + pads[0], offs[0]), padded(b, n + pads[1], offs[1]), padded(c0, n + pads[2], offs[2])
    if beta == 0.0:
        C.fill_(float("nan"))
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    B.grouped_wgrad(A, Bm, offsets, C=C, alpha=alpha, beta=beta)
    st, detail = B.sgemm_poll_device_status(torch.cuda.current_stream().cuda_stream)
    assert st == 0, detail
    ad, bd, cd = a.cuda().double(), b.cuda().double(), c0.cuda().double()
    for i in range(e):
        sl = slice(bounds[i], bounds[i + 1])
        ref = alpha * (ad[sl].mT @ bd[sl]) + (beta * cd[i] if beta else 0.0)
        if ints:
            assert torch.equal(C[i], ref.to(out)), f"group {i}"
        else:
            mag = abs(alpha) * (ad[sl].mT.abs() @ bd[sl].abs()) + abs(beta) * cd[i].abs()
            assert_close(C[i], ref, mag, additions(counts[i], t, out))
    return C


ALL = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "bf16"), ("f32", "f32")]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("t,out", ALL)
@pytest.mark.parametrize("ints", [True, False])
def test_rows_types(op, t, out, ints):
    run_rows(op, TYPES[t], TYPES[out], [5, 0, 130, 1, 64], 200, 152, ints=ints)


@pytest.mark.parametrize("t,out", ALL)
@pytest.mark.parametrize("ints", [True, False])
def test_wgrad_types(t, out, ints):
    run_wgrad(TYPES[t], TYPES[out], [5, 0, 130, 1, 64, 15, 16, 17], 136, 200, ints=ints)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [3, 0, 0], [31, 33], [127, 129, 128], [255, 257], [700]])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 64), (127, 63), (129, 65), (264, 200)])
def test_rows_sizes(t, counts, n, k):
    for op in ("T", "N"):
        run_rows(op, TYPES[t], TYPES[t], counts, n, k, ints=True, seed=n + k)


@pytest.mark.parametrize("t", ["f16", "f32"])
@pytest.mark.parametrize("counts", [[1], [0, 2, 0], [15, 33, 47], [63, 64, 65], [300]])
@pytest.mark.parametrize("m,n", [(1, 1), (64, 129), (65, 127), (257, 8), (130, 264)])
def test_wgrad_sizes(t, counts, m, n):
    run_wgrad(TYPES[t], TYPES[t], counts, m, n, ints=True, lead=3, tail=5, seed=m + n)


@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("alpha,beta", [(1.25, 0.0), (1.0, 1.0), (0.0, -0.5), (0.5, 3.0)])
def test_alpha_beta(t, out, alpha, beta):
    run_rows("T", TYPES[t], TYPES[out], [9, 70], 72, 136, alpha=alpha, beta=beta, lead=2, tail=3)
    run_wgrad(TYPES[t], TYPES[out], [9, 0, 70], 72, 136, alpha=alpha, beta=beta)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("pads,offs", [((3, 5, 7), (0, 0, 0)), ((0, 0, 0), (1, 3, 1)), ((8, 16, 8), (8, 8, 8)),
                                       ((1, 0, 0), (0, 1, 2))])
def test_strides_and_alignment(t, pads, offs):
    for op in ("T", "N"):
        run_rows(op, TYPES[t], TYPES[t], [33, 2, 100], 77, 96, ints=True, pads=pads, offs=offs, lead=1, tail=2)
    run_wgrad(TYPES[t], TYPES[t], [33, 2, 100], 77, 96, ints=True, pads=pads, offs=offs, lead=1, tail=2)


@pytest.mark.parametrize("t,out", ALL)
def test_long_sums(t, out):
    # few tiles: every tile's sum is cut over several CTAs
    run_rows("T", TYPES[t], TYPES[out], [3, 20], 256, 4096, seed=5)
    run_wgrad(TYPES[t], TYPES[out], [2500, 1596], 128, 96, seed=6)
    run_rows("N", TYPES[t], TYPES[out], [3, 20], 256, 4095, ints=True, seed=5)
    run_wgrad(TYPES[t], TYPES[out], [2500, 1, 1595], 128, 96, ints=True, seed=6)


def test_many_groups_and_a_second_call():
    rng = np.random.default_rng(3)
    counts = rng.multinomial(3000, rng.dirichlet(np.full(1024, 0.3))).tolist()
    run_rows("T", torch.bfloat16, torch.bfloat16, counts, 40, 48, ints=True)
    run_rows("T", torch.bfloat16, torch.bfloat16, counts[::-1], 40, 48, ints=True)
    run_wgrad(torch.bfloat16, torch.float32, counts, 24, 40, ints=True)


def test_larger_than_one_wave():
    counts = [700, 1, 0, 2000, 33]
    run_rows("T", torch.bfloat16, torch.bfloat16, counts, 2056, 328, ints=True)
    run_rows("N", torch.float32, torch.float32, counts, 1032, 136, ints=True)
    run_wgrad(torch.bfloat16, torch.float32, counts, 1032, 1000, ints=True)


def test_same_bits_every_time():
    x, w = values((40, 4096), torch.bfloat16, 1).cuda(), values((3, 256, 4096), torch.bfloat16, 2).cuda()
    off = torch.tensor([0, 7, 7, 40], dtype=torch.int32, device="cuda")
    first = B.grouped_gemm(x, w, off, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(B.grouped_gemm(x, w, off, out_dtype=torch.float32), first)


def test_offsets_outside_the_rows_are_clamped():
    x, w = values((50, 64), torch.bfloat16, 1, True).cuda(), values((3, 32, 64), torch.bfloat16, 2, True).cuda()
    off = torch.tensor([-7, 20, 10, 1 << 30], dtype=torch.int32, device="cuda")
    y = torch.full((50, 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.grouped_gemm(x, w, off, Y=y)
    want = torch.cat([x[:10].float() @ w[0].float().mT, torch.zeros(10, 32, device="cuda"),
                      x[20:].float() @ w[2].float().mT])
    assert torch.equal(y[:10].float(), want[:10]) and torch.equal(y[20:].float(), want[20:])


def test_neighbours_non_finite_rows_stay_out():
    """NaN and infinities in one group's rows, or weights, reach no other group."""
    for t in (torch.bfloat16, torch.float32):
        x, w = values((60, 72), t, 1, True).cuda(), values((3, 40, 72), t, 2, True).cuda()
        off = torch.tensor([0, 21, 42, 60], dtype=torch.int32, device="cuda")
        want, wantg = B.grouped_gemm(x, w, off), B.grouped_wgrad(x, x, off)
        bad, badw = x.clone(), w.clone()
        bad[21:42] = float("nan")
        bad[25] = float("inf")
        badw[1] = float("inf")
        got, gotg = B.grouped_gemm(bad, badw, off), B.grouped_wgrad(bad, bad, off)
        assert torch.equal(got[:21], want[:21]) and torch.equal(got[42:], want[42:])
        assert torch.equal(gotg[0], wantg[0]) and torch.equal(gotg[2], wantg[2])
        assert not bool(got[21:42].isfinite().any()) and bool(gotg[1].isnan().all())


def test_gradients_against_differences():
    """L = sum(Y * G) is linear in X and in W, so a central difference of any
    step gives the derivative up to the rounding of L."""
    counts, n, k = [3, 0, 5], 24, 16
    off = torch.tensor(bounds_of(counts), dtype=torch.int32, device="cuda")
    x, w, g = (values(s, torch.float32, i).cuda() for i, s in enumerate([(8, k), (3, n, k), (8, n)]))
    dx = B.grouped_gemm(g, w, off, op="N")
    dw = B.grouped_wgrad(g, x, off)

    def loss(x, w):
        return float((B.grouped_gemm(x, w, off).double() * g.double()).sum())

    h = 0.5
    for i, j in [(0, 0), (2, 15), (3, 7), (7, 3)]:
        d = torch.zeros_like(x)
        d[i, j] = h
        want = (loss(x + d, w) - loss(x - d, w)) / (2 * h)
        assert abs(float(dx[i, j]) - want) < 2e-4
    for e, i, j in [(0, 0, 0), (0, 23, 15), (1, 4, 4), (2, 11, 2)]:
        d = torch.zeros_like(w)
        d[e, i, j] = h
        want = (loss(x, w + d) - loss(x, w - d)) / (2 * h)
        assert abs(float(dw[e, i, j]) - want) < 2e-4


def test_other_stream_and_graph():
    x, w = values((40, 512), torch.bfloat16, 1).cuda(), values((4, 96, 512), torch.bfloat16, 2).cuda()
    off = torch.tensor([0, 7, 7, 30, 40], dtype=torch.int32, device="cuda")
    want = B.grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.zeros_like(want)
    B.grouped_gemm(x, w, off, Y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            B.grouped_gemm(x, w, off, Y=y)
    # new inputs and new group bounds, same graph
    x.copy_(values((40, 512), torch.bfloat16, 9))
    off.copy_(torch.tensor([0, 1, 20, 22, 40], dtype=torch.int32))
    want = B.grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


FORMS = [(16, 1), (32, 1), (64, 1), (128, 1), (256, 1), (256, 2)]


@pytest.fixture
def tile(request):
    assert B.sgemm_grouped_set_tile(*request.param) == 0
    yield request.param
    assert B.sgemm_grouped_set_tile(0) == 0


@pytest.mark.parametrize("tile", FORMS, indirect=True, ids=str)
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_every_tile(tile, t):
    """Every built tile, on ragged groups of a few and of many tiles (whole
    tiles, and tiles cut along k), with odd edges."""
    for counts, n, k in [([3, 0, 300, 17], 264, 200), ([40], 130, 4100), ([900, 0, 1, 1500, 31], 1500, 136)]:
        for op in ("T", "N"):
            run_rows(op, TYPES[t], torch.float32, counts, n, k, ints=True, lead=1, tail=2, seed=k)
    for counts, m, n in [([3, 0, 300, 17], 264, 200), ([5000, 31], 130, 140), ([900, 0, 1, 1500, 31], 700, 1000)]:
        run_wgrad(TYPES[t], torch.float32, counts, m, n, ints=True, lead=1, tail=2, seed=m)


def test_set_tile_refuses():
    for width, ctas in [(8, 1), (16, 2), (128, 2), (512, 1), (-1, 1), (64, 3)]:
        assert B.sgemm_grouped_set_tile(width, ctas) == B.SGEMM_ERR_INVALID_VALUE


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("k", [96, 91])
def test_one_matrix_for_every_group(t, op, k):
    x, w = values((50, k), TYPES[t], 1, True).cuda(), values((40, k) if op == "T" else (k, 40), TYPES[t], 2, True).cuda()
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda")
    y = B.grouped_gemm(x, w.expand(3, *w.shape), off, op=op)
    assert torch.equal(y.float(), x.float() @ (w.float().mT if op == "T" else w.float()))


def test_from_a_new_host_thread():
    """A thread whose first CUDA work is the call (as autograd's is)."""
    import threading
    x, w = values((40, 64), torch.bfloat16, 1).cuda(), values((2, 32, 64), torch.bfloat16, 2).cuda()
    off = torch.tensor([0, 7, 40], dtype=torch.int32, device="cuda")
    want = B.grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    y = torch.zeros_like(want)
    s = torch.cuda.current_stream().cuda_stream
    args = (B.SGEMM_OP_T, B.SGEMM_TYPE_BF16, B.SGEMM_TYPE_BF16, 2, 40, 32, 64, 1.0, x.data_ptr(), 64, w.data_ptr(),
            64, 32 * 64, off.data_ptr(), 0.0, y.data_ptr(), 32, s)
    got = []
    t = threading.Thread(target=lambda: got.append(B.sgemm_grouped(*args)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == [0] and torch.equal(y, want)


def test_overlapping_groups_take_each_row_once():
    """Bounds that no caller means: every row belongs to the first group that
    has it, however many claim it."""
    e, t = 1024, 500
    x, w = values((t, 32), torch.bfloat16, 1, True).cuda(), values((e, 24, 32), torch.bfloat16, 2, True).cuda()
    off = torch.tensor([0, t] * (e // 2) + [0], dtype=torch.int32, device="cuda")
    y = B.grouped_gemm(x, w, off)
    assert torch.equal(y.float(), x.float() @ w[0].float().mT)
    dw = B.grouped_wgrad(y, x, off, out_dtype=torch.float32)
    assert torch.equal(dw[0], y.float().mT @ x.float()) and not bool(dw[1:].any())


def test_fp32_operands_up_to_the_largest():
    """Values beyond BF16's largest, and the smallest normal ones, keep their bits."""
    most = torch.finfo(torch.float32).max
    x = torch.tensor([[most, -most, 3.39e38, 1.2e-38]], device="cuda")
    w = torch.eye(4, device="cuda") * 0.5
    y = B.grouped_gemm(x, w[None].contiguous(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[0, :3], x[0, :3] * 0.5)
    assert abs(float(y[0, 3]) - 0.6e-38) < 1e-40


def test_shares_the_workspace_with_the_other_products():
    """Split-K flags, partial tiles and counters of one stream, call after call."""
    a, b = values((256, 8192), torch.float32, 1, True).cuda(), values((8192, 256), torch.float32, 2, True).cuda()
    want = (a.double() @ b.double()).float()
    xb, off = a.bfloat16(), torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    wb = b.mT.contiguous().bfloat16()[None].expand(2, 256, 8192)
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        for call in (B.sgemm, B.sgemm_3xtf32):
            c = torch.empty(256, 256, device="cuda")
            assert call(256, 256, 8192, 1.0, a.data_ptr(), 8192, b.data_ptr(), 256, 0.0, c.data_ptr(), 256, s) == 0
            y = B.grouped_gemm(xb, wb, off, out_dtype=torch.float32)
            assert torch.equal(c, want) and torch.equal(y, want)
    assert B.sgemm_poll_device_status(s)[0] == 0


def test_capture_needs_the_workspace():
    x, w = values((40, 64), torch.bfloat16, 1).cuda(), values((2, 32, 64), torch.bfloat16, 2).cuda()
    off = torch.tensor([0, 7, 40], dtype=torch.int32, device="cuda")
    y = torch.zeros(40, 32, dtype=torch.bfloat16, device="cuda")
    want = B.grouped_gemm(x, w, off)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(B.SgemmError) as e:
                B.grouped_gemm(x, w, off, Y=y)
    assert e.value.status == B.SGEMM_ERR_CAPTURE
    B.grouped_gemm(x, w, off, Y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["T", "N"])
def test_copied_rows_from_every_address(t, op):
    """Operands at every element offset and pitch within 16 bytes, rows that end inside a copied piece."""
    for r in range(8):
        run_rows(op, TYPES[t], TYPES[t], [20, 0, 45], 61 + r, 500 + 3 * r, ints=True,
                 pads=(r, (3 * r) % 8, r % 3), offs=(r, 7 - r, 0))


@pytest.mark.parametrize("tile", FORMS, indirect=True, ids=str)
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[300, 20, 0, 700, 65, 128, 1, 300], [3000, 1, 1, 1, 64, 2, 2], [5, 900, 901, 3],
                                    list(range(0, 130, 2)) + [1000] + [1] * 70], ids=len)
def test_wgrad_many_tiles_of_different_lengths(tile, t, counts):
    """More tiles than the workers of any form, groups of very different lengths: every element once, whoever adds it."""
    m, n = (1030, 2050) if len(counts) < 50 else (130, 264)
    run_wgrad(TYPES[t], torch.float32, counts, m, n, ints=True)
