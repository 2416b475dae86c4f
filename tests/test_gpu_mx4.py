"""4-bit floating point in blocks of 32: the rounding, bit by bit, and the product
against the rounded values in 64 bits.

Tolerance of the product. Each product of two codes and their powers is exact.
The tensor core truncates its sums: n instructions of 64 values put one result at
most n * 2^-23 of the sum of magnitudes off (n at most 32 for FP32 results, 128
for others, then sums in FP32); the result is rounded to its type."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24
VALUES = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def rounding(want, t):
    f = torch.finfo(t)
    return torch.maximum(want.abs() * f.eps / 2, torch.full_like(want, f.smallest_normal * f.eps / 2))


def untile(scale, rows, blocks):
    """The scales as (rows, blocks)."""
    t = scale.view(-(-rows // 128), -(-blocks // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-(-rows // 128) * 128, -1)[:rows, :blocks]


def values(q, scale, rows):
    """What codes and scales stand for, in 64 bits."""
    blocks = q.shape[1] // 16
    codes = torch.stack([q & 15, q >> 4], dim=2).view(rows, -1).long()
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=q.device)
    powers = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [float("nan")], dtype=torch.float64, device=q.device)
    s = powers[untile(scale, rows, blocks).long()]
    return (table[codes].view(rows, blocks, 32) * s[:, :, None]).view(rows, -1)


def rounded(x):
    """(codes, biased powers) by the definition, on the CPU in 64 bits."""
    rows, k = x.shape
    blocks = -(-k // 32)
    v = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    v[:, :k] = x.double().cpu()
    v = v.view(rows, blocks, 32)
    most = v.abs().amax(dim=2)
    power = (torch.frexp(most).exponent - 3).clamp(min=-127)
    power = torch.where(most > 0, power, -127)
    a = v.abs() / torch.pow(2.0, power.double())[:, :, None]
    code = torch.zeros_like(v)
    # ties go to the even code: up at the borders below an even one
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5, False)):
        code += (a >= border) if up else (a > border)
    # (codes 0 to 7 are the values in their order)
    return (code.long() + 8 * torch.signbit(v).long()).view(rows, -1), (power + 127)


SIZES = [(1, 1), (1, 32), (3, 33), (5, 64), (133, 1000), (128, 4096), (129, 130), (300, 777), (1, 5000)]


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_rounding(t, m, k):
    x = rand(m, k, seed=m + k)
    x *= torch.pow(2.0, rand(m, 1, seed=3, scale=4.0).round())
    x[:, :: 37] = 0
    x = x.to(t)
    q, s = B.mx4_quantize(x)
    code, power = rounded(x)
    blocks = power.shape[1]
    assert q.shape == (m, 16 * blocks) and s.numel() == -(-m // 128) * -(-blocks // 4) * 512
    got = torch.stack([q & 15, q >> 4], dim=2).view(m, -1).long().cpu()
    assert torch.equal(got, code)
    assert torch.equal(untile(s, m, blocks).long().cpu(), power.long())
    assert torch.equal(B.mx4_tile_scales(power.to(torch.uint8).cuda()), s)     # zeros elsewhere
    for out in TYPES:
        back = B.mx4_dequantize(q, s, k, out_dtype=out)
        assert back.dtype == out and torch.equal(back, values(q, s, m)[:, :k].to(out))


@pytest.mark.parametrize("m,k,offset,pad", [(300, 1001, 0, 0), (1000, 33, 1, 0), (257, 4097, 3, 2), (64, 2045, 2, 3),
                                            (50, 8191, 5, 8), (2000, 3, 0, 0), (1, 1027, 7, 0), (130, 1024, 4, 1), (9, 96, 6, 0)])
@pytest.mark.parametrize("t", TYPES)
def test_rows_that_start_anywhere(t, m, k, offset, pad):
    """The codes of the same rows, aligned; back into rows that start anywhere, and nothing beside them."""
    x = rand(m, k, seed=m + k)
    x *= torch.pow(2.0, rand(m, k, seed=3, scale=2.0).round())
    x = x.to(t)
    x[m // 2, k // 2] = float("inf")
    whole = torch.zeros(m, (k + 7) // 8 * 8, dtype=t, device="cuda")
    whole[:, :k] = x
    want, want_scale = B.mx4_quantize(whole)                     # (zeros behind the row: the same blocks)
    nan = float("nan")
    store = torch.full((offset + m * (k + pad) + 8,), nan, dtype=t, device="cuda")
    view = store[offset:offset + m * (k + pad)].view(m, k + pad)[:, :k]
    view.copy_(x)
    q, scale = B.mx4_quantize(view)
    assert torch.equal(q, want) and torch.equal(scale, want_scale)
    view.fill_(7)
    back = B.mx4_dequantize(q, scale, k, X=view)
    assert back is view
    assert torch.equal(view.nan_to_num(nan=1e4), values(q, scale, m)[:, :k].to(t).nan_to_num(nan=1e4))
    beside = store[offset:offset + m * (k + pad)].view(m, k + pad)[:, k:]
    assert bool(store[:offset].isnan().all()) and bool(beside.isnan().all()) and bool(store[offset + m * (k + pad):].isnan().all())


def test_borders():
    """Every border between two values, and its neighbours, in blocks of several powers."""
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.99]
    for t in TYPES:
        e = torch.finfo(t).eps
        near = [b * f for b in borders for f in (1 - e, 1, 1 + e)]
        row = torch.tensor(near[:27] + [7.5, 0.0, -0.0, 6.0, -7.5], dtype=torch.float64)
        x = torch.stack([row * 2.0 ** p for p in (-10, -3, 0, 5, 9)] + [-row]).to(t).cuda()
        q, s = B.mx4_quantize(x)
        code, power = rounded(x)
        got = torch.stack([q & 15, q >> 4], dim=2).view(x.shape[0], -1).long().cpu()
        assert torch.equal(got, code) and torch.equal(untile(s, 6, 1).long().cpu(), power.long())


def test_extremes():
    for t in TYPES:
        f = torch.finfo(t)
        x = torch.zeros(6, 64, dtype=t, device="cuda")
        x[0, 0], x[0, 40] = f.max, f.smallest_normal * f.eps
        x[1, 3] = float("nan")
        x[2, 3] = float("inf")
        x[3, 3], x[3, 35] = float("-inf"), 1.0
        x[4, 0] = -f.smallest_normal
        q, s = B.mx4_quantize(x)
        sc = untile(s, 6, 2).long().cpu()
        want = rounded(torch.where(x.isfinite(), x, torch.zeros_like(x)))[1].long()
        want[1, 0] = want[2, 0] = want[3, 0] = 255
        assert torch.equal(sc, want)
        back = B.mx4_dequantize(q, s, 64, out_dtype=torch.float32)
        nan = torch.zeros(6, 64, dtype=torch.bool)
        nan[1:4, :32] = True
        assert torch.equal(back.isnan().cpu(), nan)
        assert torch.equal(back[~nan.cuda()].double(), values(q, s, 6)[~nan.cuda()].float().double())


def product(m, n, k, out, seed=0, spread=3.0):
    a = rand(m, k, seed=seed) * torch.pow(2.0, rand(m, 1, seed=seed + 2, scale=spread).round())
    b = rand(n, k, seed=seed + 1) * torch.pow(2.0, rand(1, k, seed=seed + 3, scale=spread).round())
    if out == torch.float16:
        a, b = a * 0.01, b * 0.01
    qa, sa = B.mx4_quantize(a.bfloat16())
    qb, sb = B.mx4_quantize(b.bfloat16())
    return qa, sa, qb, sb


def check(c, qa, sa, qb, sb, k):
    va, vb = values(qa, sa, qa.shape[0]), values(qb, sb, qb.shape[0])
    want = va @ vb.mT
    n = min(-(-k // 64), 32 if c.dtype == torch.float32 else 128) + -(-k // 2048)
    slack = (va.abs() @ vb.abs().mT) * n * 2.0 ** -23 + rounding(want, c.dtype)
    off = (c.double() - want).abs() - slack
    assert bool((off <= 0).all()), f"off by {float(off.max()):.3g} more than allowed"


PRODUCTS = [(1, 1, 1), (1, 4096, 4096), (7, 130, 70), (16, 300, 256), (17, 300, 512), (33, 500, 1000), (64, 129, 320),
            (65, 128, 64), (133, 8191, 1000), (128, 256, 2080), (200, 70, 5000), (257, 513, 777), (1000, 1100, 520),
            (2, 100, 20000), (300, 520, 17000)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("out", TYPES)
def test_product(out, m, n, k):
    ops = product(m, n, k, out)
    c = B.mx4_gemm(*ops, out_dtype=out)
    assert c.dtype == out and c.shape == (m, n)
    check(c, *ops, k)


@pytest.mark.parametrize("tile", [(16, 1), (32, 1), (64, 1), (128, 1), (256, 1), (256, 2)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_every_tile(tile, out):
    """Every built form: cut along k and whole, several accumulations, ragged in each size; small integers are exact."""
    width = tile[0]
    sizes = [(min(width, 100), 300, 1000), (width, 20000, 256), (min(width, 99), 130, 9000)]
    if width >= 128:
        sizes += [(width + 1, 257, 800), (3 * width + 70, 400, 4500), (5000, 3000, 96)]
    try:
        assert B.sgemm_grouped_set_tile(*tile) == 0
        for m, n, k in sizes:
            ops = product(m, n, k, out)
            c = B.mx4_gemm(*ops, out_dtype=out)
            assert f"x{width}x" in B.sgemm_last_config() and f"cluster={tile[1]}" in B.sgemm_last_config()
            check(c, *ops, k)
            g = torch.Generator(device="cuda").manual_seed(1)
            a = torch.randint(-1, 2, (m, k), generator=g, device="cuda").float()
            b = torch.randint(-1, 2, (n, k), generator=g, device="cuda").float()
            c = B.mx4_gemm(*B.mx4_quantize(a), *B.mx4_quantize(b), out_dtype=torch.float32)
            assert torch.equal(c.double(), a.double() @ b.double().mT)
    finally:
        B.sgemm_grouped_set_tile(0)


def test_scales_that_are_none():
    m, n, k = 40, 200, 512
    qa, sa, qb, sb = product(m, n, k, torch.float32)
    x = rand(m, k).bfloat16()
    x[5, 100] = float("nan")
    w = rand(n, k, seed=1).bfloat16()
    w[7, 300] = float("inf")
    c = B.mx4_gemm(*B.mx4_quantize(x), *B.mx4_quantize(w), out_dtype=torch.float32)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[5], bad[:, 7] = True, True
    assert torch.equal(c.isnan(), bad)


@pytest.mark.parametrize("out", TYPES)
def test_strides_and_guards(out):
    m, n, k = 37, 203, 300
    qa, sa, qb, sb = product(m, n, k, out)
    want = B.mx4_gemm(qa, sa, qb, sb, out_dtype=out)
    pad = torch.full((m, qa.shape[1] + 32), 255, dtype=torch.uint8, device="cuda")
    pad[:, : qa.shape[1]] = qa
    store = torch.full((m * (n + 5) + 8,), 77.0, dtype=out, device="cuda")
    view = store[1: 1 + m * (n + 5)].view(m, n + 5)[:, :n]
    c = B.mx4_gemm(pad[:, : qa.shape[1]], sa, qb, sb, C=view)
    assert c is view and torch.equal(view, want)
    mask = torch.ones(store.numel(), dtype=torch.bool, device="cuda")
    mask[1: 1 + m * (n + 5)].view(m, n + 5)[:, :n] = False
    assert bool((store[mask] == 77).all())
    # the quantiser: rows at any element, codes with a pitch of their own
    x = rand(m, k, seed=9).to(out)
    q0, s0 = B.mx4_quantize(x)
    wide = torch.zeros(m * (k + 3) + 1, dtype=out, device="cuda")
    xv = wide[1:].view(m, k + 3)[:, :k]
    xv.copy_(x)
    pad.fill_(7)
    q, s = B.mx4_quantize(xv, Q=pad[:, : q0.shape[1]])
    assert torch.equal(pad[:, : q0.shape[1]], q0) and torch.equal(s, s0) and bool((pad[:, q0.shape[1]:] == 7).all())
    back = torch.full((m * (k + 3) + 1,), 77.0, dtype=out, device="cuda")
    bv = back[1:].view(m, k + 3)[:, :k]
    assert B.mx4_dequantize(q0, s0, k, X=bv) is bv
    assert torch.equal(bv, B.mx4_dequantize(q0, s0, k, out_dtype=out)) and bool((back[1:].view(m, k + 3)[:, k:] == 77).all())


def test_empty():
    for t in TYPES:
        q, s = B.mx4_quantize(torch.zeros(0, 64, dtype=t, device="cuda"))
        assert q.shape == (0, 32) and s.numel() == 0
        qb, sb = B.mx4_quantize(rand(5, 64).to(t))
        assert B.mx4_gemm(q, s, qb, sb).shape == (0, 5) and B.mx4_gemm(qb, sb, q, s).shape == (5, 0)
        q, s = B.mx4_quantize(torch.zeros(3, 0, dtype=t, device="cuda"))
        c = B.mx4_gemm(q, s, *B.mx4_quantize(torch.zeros(4, 0, dtype=t, device="cuda")))
        assert c.shape == (3, 4) and not bool(c.any())
        assert B.mx4_dequantize(q, s, 0).shape == (3, 0)


def test_same_bits_each_time_and_on_another_stream():
    for m, n, k in ((3, 1000, 4096), (700, 900, 2048)):
        ops = product(m, n, k, torch.float32)
        first = B.mx4_gemm(*ops, out_dtype=torch.float32)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        second = B.mx4_gemm(*ops, out_dtype=torch.float32, stream=other)
        torch.cuda.current_stream().wait_stream(other)
        for _ in range(5):
            assert torch.equal(first, B.mx4_gemm(*ops, out_dtype=torch.float32))
        assert torch.equal(first, second)


def test_captured():
    m, n, k = 20, 600, 4096
    x, w = rand(m, k).bfloat16(), rand(n, k, seed=1).bfloat16()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qw, sw = B.mx4_quantize(w)
        B.mx4_gemm(*B.mx4_quantize(x), qw, sw)          # sizes the stream's workspace
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                  # two graphs that share it
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c = B.mx4_gemm(*B.mx4_quantize(x), qw, sw)
        graphs.append((graph, c))
    for seed in (3, 4):
        x.copy_(rand(m, k, seed=seed))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = B.mx4_gemm(*B.mx4_quantize(x), qw, sw)
        assert all(torch.equal(c, want) for _, c in graphs)


def test_capture_needs_the_workspace():
    ops, x = product(8, 100, 64, torch.bfloat16), rand(8, 64)
    torch.cuda.synchronize()
    B.sgemm_shutdown()                                   # no stream has one (torch hands out streams again)
    want = B.mx4_gemm(*ops)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(B.SgemmError) as e:
        with torch.cuda.graph(graph, stream=side):
            B.mx4_quantize(x)                             # (has no need of one)
            B.mx4_gemm(*ops)
    assert e.value.status == B.SGEMM_ERR_CAPTURE
    torch.cuda.synchronize()
    assert torch.equal(B.mx4_gemm(*ops, stream=side), want)


def test_norm_into_the_4_bit_product():
    """A layer as it is served: norm, 4 bits, product."""
    x, r = rand(50, 640).bfloat16(), rand(50, 640, seed=1).bfloat16()
    y, h, _ = B.rms_norm(x, (1 + 0.1 * rand(640, seed=2)), residual=r)
    qw, sw = B.mx4_quantize(rand(300, 640, seed=3, scale=0.04).bfloat16())
    q, s = B.mx4_quantize(y)
    check(B.mx4_gemm(q, s, qw, sw), q, s, qw, sw, 640)
    # against the layer without rounding: 4 bits are off by some 10 % of a value
    full = y.double() @ values(qw, sw, 300).mT
    got = B.mx4_gemm(q, s, qw, sw, out_dtype=torch.float32).double()
    assert float((got - full).norm() / full.norm()) < 0.25
