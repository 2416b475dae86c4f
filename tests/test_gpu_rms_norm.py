"""The residual's addition with the root-mean-square norm, its 8-bit form and its
gradients, against the formulas in 64 bits.

Tolerances. A rounding to type t is off by half a step, eps(t) / 2 of the value;
below the normal numbers steps are smallest_normal(t) * eps(t) whatever the
value (2^-24 for F16, whose normal numbers end at 2^-14).
FP32 parts: a sum of n terms is off by at most (terms added one after another) *
2^-24 of the sum of magnitudes; a row's longest chain is below 64 additions at
the sizes here (at most 20000 values over 512 threads in pieces, then a tree)."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from dense_fp32_gemm_gb300 import layers

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24


def rounding(want, t):
    """Half a step of type t at the values `want`."""
    f = torch.finfo(t)
    return torch.maximum(want.abs() * f.eps / 2, torch.full_like(want, f.smallest_normal * f.eps / 2))


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def inputs(m, n, t, wt, residual=True, seed=0):
    x = rand(m, n, seed=seed).to(t)
    r = rand(m, n, seed=seed + 1, scale=3.0).to(t) if residual else None
    w = (1 + 0.2 * rand(n, seed=seed + 2)).to(wt)
    return x, r, w


def reference(x, r, w, eps=1e-6):
    """h as it is stored, then (rstd, y) of it in 64 bits."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = h.double()
    rstd = 1 / (f.square().mean(dim=1) + eps).sqrt()
    return h, rstd, f * rstd[:, None] * w.double()


def close(got, want, slack):
    """|got - want| <= slack (a tensor or number), reported where it fails."""
    off = (got.double() - want).abs() - slack
    assert bool((off <= 0).all()), f"off by {float(off.max()):.3g} more than allowed"


SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (133, 1001), (300, 4096), (700, 520), (40, 16384), (6, 20000),
         (5, 5001), (2000, 136), (1, 8), (30001, 64), (9001, 128), (77, 248), (5000, 256)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_forward(t, m, n, residual):
    for wt in {t, torch.float32}:
        x, r, w = inputs(m, n, t, wt, residual)
        y, h, rstd = B.rms_norm(x, w, residual=r)
        ref_h, ref_rstd, ref_y = reference(x, r, w)
        assert h.dtype == y.dtype == t and torch.equal(h, ref_h)
        assert (h is x) == (r is None)
        # the mean (64 additions and two products) halved by the root, root and quotient
        close(rstd, ref_rstd, ref_rstd * 36 * U)
        close(y, ref_y, rounding(ref_y, t) + ref_y.abs() * 40 * U)


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_8_bits(t, m, n):
    for wt in {t, torch.float32}:
        x, r, w = inputs(m, n, t, wt)
        q, scale, h = B.rms_norm_i8(x, w, residual=r)
        ref_h, ref_rstd, _ = reference(x, r, w)
        assert torch.equal(h, ref_h)
        u = (h.double() * w.double()).float().double()
        step = (u.abs().amax(dim=1) / 127).float().double()
        want = (u / step[:, None]).float().double().round().clamp(-127, 127)
        assert torch.equal(q.double(), want)                    # defined exactly
        close(scale, step * ref_rstd, step * ref_rstd * 38 * U)


@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("t", TYPES)
def test_gradients(t, m, n, with_dh):
    for wt in {t, torch.float32}:
        x, r, w = inputs(m, n, t, wt)
        _, h, rstd = B.rms_norm(x, w, residual=r)
        dy = rand(m, n, seed=7).to(t)
        dh = rand(m, n, seed=8).to(t) if with_dh else None
        dx, dw = B.rms_norm_grad(dy, h, w, rstd, dH=dh)
        assert dx.dtype == t and dw.dtype == wt
        _, s, _ = reference(h, None, w)
        nrm = h.double() * s[:, None]
        d = dy.double() * w.double()
        mean = (d * nrm).mean(dim=1, keepdim=True)
        want = s[:, None] * (d - nrm * mean)
        # rstd is off by 36 U; the mean's 64 additions and its products' roundings
        loose = s[:, None] * (d.abs() + nrm.abs() * (d * nrm).abs().mean(dim=1, keepdim=True)) * 150 * U
        if with_dh:
            want = want + dh.double()
            loose = loose + want.abs() * U
        close(dx, want, rounding(want, t) + loose)
        want = (dy.double() * nrm).sum(dim=0)
        # a block's rows (at least 152 blocks, or a row each), 608 / 8 parts and 8 groups one after another;
        # for the longest rows the rows of a slab
        # short rows: at most 32 of them in a block add their sums to one another's
        chain = (m / (152 if n < 20000 else 1) + 1) + 76 + 8 + 40
        loose = (dy.double() * nrm).abs().sum(dim=0) * chain * U
        close(dw, want, rounding(want, wt) + loose)


def test_gradient_against_differences():
    """Along a direction, the 64-bit formula's difference quotient."""
    m, n = 17, 200
    x, r, w = inputs(m, n, torch.float32, torch.float32)
    a, b = rand(m, n, seed=5).double(), rand(m, n, seed=6).double()     # weights of y and h in a loss

    def loss(x, r, w):
        h = x + r
        y = h / (h.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * w
        return (y * a + h * b).sum()

    leaves = [v.clone().requires_grad_() for v in (x, w, r)]
    y, h = layers.rms_norm(leaves[0], leaves[1], residual=leaves[2])
    grads = torch.autograd.grad((y * a.float() + h * b.float()).sum(), leaves)
    step = 1e-5
    for i, (leaf, g) in enumerate(zip((x, w, r), grads)):
        v = rand(*leaf.shape, seed=20 + i).double()
        at = [x.double(), r.double(), w.double()]
        k = (0, 2, 1)[i]
        plus, minus = list(at), list(at)
        plus[k] = at[k] + step * v
        minus[k] = at[k] - step * v
        slope = (loss(*plus) - loss(*minus)) / (2 * step)
        got = (g.double() * v).sum()
        # the quotient's own error is some step^2 = 1e-10 of the third derivative; FP32 gradients: 200 U of the terms
        size = (g.double() * v).abs().sum()
        assert abs(float(slope - got)) <= float(size) * (200 * U + 1e-7)


def test_autograd_forms():
    x, r, w = inputs(6, 40, torch.bfloat16, torch.float32)
    x3 = x.view(2, 3, 40).clone().requires_grad_()
    y = layers.rms_norm(x3, w)
    assert y.shape == x3.shape and not w.requires_grad
    (g,) = torch.autograd.grad(y.float().sum(), [x3])
    _, h, rstd = B.rms_norm(x, w)
    want, none = B.rms_norm_grad(torch.ones_like(x), h, w, rstd, want=(True, False))
    assert none is None and torch.equal(g.view(6, 40), want)
    # only the sum is used: its gradient passes through
    xr, rr, wr = x.clone().requires_grad_(), r.clone().requires_grad_(), w.clone().requires_grad_()
    _, h = layers.rms_norm(xr, wr, residual=rr)
    gx, gw, gr = torch.autograd.grad(h.float().sum(), [xr, wr, rr])
    assert torch.equal(gx, torch.ones_like(x)) and torch.equal(gr, gx) and not bool(gw.any())
    # second derivatives are refused
    y = layers.rms_norm(xr, wr)
    (g,) = torch.autograd.grad(y.float().square().sum(), [xr], create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()
    none, dw = B.rms_norm_grad(torch.ones_like(x), *B.rms_norm(x, w)[1:2], w, B.rms_norm(x, w)[2], want=(False, True))
    assert none is None and dw.shape == w.shape


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (8, 0)])
def test_strides_and_guards(t, offset, pad):
    """Rows at any element and pitch; what lies between and behind them stays."""
    m, n = 37, 264

    def buffer(values, like=None):
        store = torch.full((offset + m * (n + pad) + 16,), 77, dtype=like or t, device="cuda")
        view = store[offset: offset + m * (n + pad)].view(m, n + pad)[:, :n]
        if values is not None:
            view.copy_(values)
        return store, view

    x, r, w = inputs(m, n, t, t)
    y0, h0, rstd0 = B.rms_norm(x, w, residual=r)
    (_, xv), (_, rv), (ys, yv), (hs, hv) = buffer(x), buffer(r), buffer(None), buffer(None)
    y, h, rstd = B.rms_norm(xv, w, residual=rv, Y=yv, H=hv)
    assert y is yv and h is hv
    assert torch.equal(hv, h0)
    close(yv, y0.double(), 2 * rounding(y0.double(), t) + y0.double().abs() * 80 * U)
    q0, s0, _ = B.rms_norm_i8(x, w, residual=r)
    qs, qv = buffer(None, torch.int8)
    q, s, _ = B.rms_norm_i8(xv, w, residual=rv, Q=qv, H=hv)
    assert torch.equal(qv, q0)
    dy, dh = rand(m, n, seed=3).to(t), rand(m, n, seed=4).to(t)
    (_, dyv), (_, dhv), (dxs, dxv) = buffer(dy), buffer(dh), buffer(None)
    dx0, dw0 = B.rms_norm_grad(dy, h0, w, rstd0, dH=dh)
    dx, dw = B.rms_norm_grad(dyv, hv, w, rstd, dH=dhv, dX=dxv)
    assert dx is dxv
    close(dxv, dx0.double(), 2 * rounding(dx0.double(), t) + 400 * U)
    for s, v in ((ys, yv), (hs, hv), (qs, qv), (dxs, dxv)):
        mask = torch.ones(s.numel(), dtype=torch.bool, device="cuda")
        mask[offset: offset + m * (n + pad)].view(m, n + pad)[:, :n] = False
        assert bool((s[mask] == 77).all())


# odd rows, many of them to a block; the longest that registers hold, and longer
ODD = [(2000, 1001), (3000, 333), (700, 4097), (3000, 255), (30001, 65), (5000, 3), (170, 8191), (200, 8185), (9, 16377),
       (165, 16383), (6, 20001)]


@pytest.mark.parametrize("m,n", ODD)
@pytest.mark.parametrize("t", TYPES)
def test_rows_that_start_anywhere(t, m, n):
    test_forward(t, m, n, True)
    test_8_bits(t, m, n)
    test_gradients(t, m, n, True)


# rows that the registers of a block hold, and those that they do not (at
# most 35 pieces of 4 values a thread: 35 + 4 + 21 additions one after another)
@pytest.mark.parametrize("m,n", [(1000, 8192), (333, 5120), (400, 12288), (90, 16384), (50, 20000), (30, 32768), (5, 70000)])
@pytest.mark.parametrize("t", TYPES)
def test_long_rows(t, m, n):
    test_forward(t, m, n, True)
    test_gradients(t, m, n, True)
    test_gradients(t, m, n, False)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,offset,pads", [(333, 5, (2, 2, 2, 2)), (333, 5, (2, 10, 18, 2)), (333, 2, (2, 3, 2, 2)),
                                           (40, 1, (1, 1, 1, 1)), (40, 1, (0, 0, 0, 8)), (2048, 4, (8, 8, 8, 16)),
                                           (5001, 1, (0, 1, 0, 0))])
def test_many_rows_at_any_pitch(t, n, offset, pads):
    """Matrices that start alike after a 16-byte boundary, and not."""
    m = 1500

    def at(values, pad):
        store = torch.full((offset + m * (n + pad),), 77, dtype=values.dtype, device="cuda")
        view = store[offset:].view(m, n + pad)[:, :n]
        view.copy_(values)
        return store, view

    x, r, w = inputs(m, n, t, t)
    ref_h, ref_rstd, ref_y = reference(x, r, w)
    empty = torch.zeros_like(x)
    stores, views = zip(*(at(v, p) for v, p in zip((x, r, empty, empty), pads)))
    y, h, rstd = B.rms_norm(views[0], w, residual=views[1], Y=views[2], H=views[3])
    assert torch.equal(h, ref_h)
    close(rstd, ref_rstd, ref_rstd * 36 * U)
    close(y, ref_y, rounding(ref_y, t) + ref_y.abs() * 40 * U)
    q, scale, _ = B.rms_norm_i8(views[0], w, residual=views[1], H=views[3])
    q0, scale0, _ = B.rms_norm_i8(x, w, residual=r)
    assert torch.equal(q, q0)
    close(scale, scale0.double(), scale0.double() * 76 * U)          # two of 38 U
    dy, dh = rand(m, n, seed=7).to(t), rand(m, n, seed=8).to(t)
    views[0].copy_(dy), views[1].copy_(dh)
    dx, dw = B.rms_norm_grad(views[0], h, w, rstd, dH=views[1], dX=views[2])
    _, s, _ = reference(h, None, w)
    nrm, d = h.double() * s[:, None], dy.double() * w.double()
    mean = (d * nrm).mean(dim=1, keepdim=True)
    want = s[:, None] * (d - nrm * mean) + dh.double()
    loose = s[:, None] * (d.abs() + nrm.abs() * (d * nrm).abs().mean(dim=1, keepdim=True)) * 150 * U + want.abs() * U
    close(dx, want, rounding(want, t) + loose)                       # as in test_gradients
    want = (dy.double() * nrm).sum(dim=0)
    chain = (m / 152 + 1) + 76 + 8 + 40
    close(dw, want, rounding(want, t) + (dy.double() * nrm).abs().sum(dim=0) * chain * U)
    for store, pad in zip(stores, pads):
        assert bool((store[:offset] == 77).all()) and bool((store[offset:].view(m, n + pad)[:, n:] == 77).all())


def test_in_place():
    for n in (64, 520, 20000, 5001):
        x, r, w = inputs(9, n, torch.bfloat16, torch.bfloat16)
        y0, h0, rstd0 = B.rms_norm(x, w, residual=r)
        x1, r1 = x.clone(), r.clone()
        version = r1._version
        y, h, rstd = B.rms_norm(x1, w, residual=r1, Y=x1, H=r1)     # the sum stays in the residual's place
        assert y is x1 and h is r1 and r1._version > version
        assert torch.equal(x1, y0) and torch.equal(r1, h0) and torch.equal(rstd, rstd0)
        dy, dh = rand(9, n, seed=3).bfloat16(), rand(9, n, seed=4).bfloat16()
        dx0, dw0 = B.rms_norm_grad(dy, h0, w, rstd0, dH=dh)
        for place in (0, 1, 2):
            given = [dy.clone(), h0.clone(), dh.clone()]
            dx, dw = B.rms_norm_grad(given[0], given[1], w, rstd0, dH=given[2], dX=given[place])
            assert dx is given[place] and torch.equal(dx, dx0) and torch.equal(dw, dw0)


@pytest.mark.parametrize("n", [96, 600])
def test_no_numbers_and_extremes(n):
    for t in TYPES:
        big = torch.finfo(t).max
        x = rand(8, n).to(t)
        x[0] = 0
        x[1, 5] = float("nan")
        x[2, 7] = float("inf")
        x[3, 7], x[3, 8] = float("inf"), float("nan")
        x[4] = big / 4                  # the squares' sum is beyond FP32 for two of the types
        x[5] = torch.finfo(t).tiny
        w = torch.ones(n, dtype=t, device="cuda")
        y, _, rstd = B.rms_norm(x, w)
        f = x.double()
        ref = 1 / (f.square().mean(dim=1) + 1e-6).sqrt()
        assert not bool(y[0].any())
        assert bool(y[1].isnan().all()) and bool(y[3].isnan().all())
        assert bool(y[2, 7].isnan()) and not bool(y[2, :7].any())
        rows = [0, 4, 5, 6, 7]
        # (a factor below FP32's normal numbers is stored with an error of 2^-150)
        close(rstd[rows], ref[rows], ref[rows] * 36 * U + 2.0 ** -149)
        want = f * ref[:, None]
        close(y[rows], want[rows], rounding(want[rows], t) + want[rows].abs() * 40 * U)
        q, scale, _ = B.rms_norm_i8(x, w)
        assert float(scale[0]) == 0 and not bool(q[:4].any())
        assert bool(scale[1:4].isnan().all())
        assert bool((q[4] == 127).all()) and abs(float(scale[4]) * 127 - 1) < 1e-5
        # the sum overflows its type: an infinity, as the addition gives
        _, h, _ = B.rms_norm(x[4:5], w, residual=torch.full_like(x[4:5], big))
        assert bool(h.isinf().all())


def test_empty():
    w = torch.ones(8, device="cuda")
    x = torch.zeros(0, 8, device="cuda")
    y, h, rstd = B.rms_norm(x, w)
    assert y.shape == (0, 8) and rstd.shape == (0,)
    dx, dw = B.rms_norm_grad(x, h, w, rstd)
    assert dx.shape == (0, 8) and not bool(dw.any())
    y, _, _ = B.rms_norm(torch.zeros(3, 0, device="cuda"), torch.ones(0, device="cuda"))
    assert y.shape == (3, 0)


def test_same_bits_each_time_and_on_another_stream():
    x, r, w = inputs(3000, 1000, torch.bfloat16, torch.float32)
    dy = rand(3000, 1000, seed=9).bfloat16()

    def all_of(stream=None):
        y, h, rstd = B.rms_norm(x, w, residual=r, stream=stream)
        q, s, _ = B.rms_norm_i8(x, w, residual=r, stream=stream)
        return (y, h, rstd, q, s) + B.rms_norm_grad(dy, h, w, rstd, stream=stream)

    first = all_of()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    second = all_of(other)
    torch.cuda.current_stream().wait_stream(other)
    third = all_of()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured():
    x, r, w = inputs(64, 2048, torch.bfloat16, torch.bfloat16)
    dy = rand(64, 2048, seed=9).bfloat16()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, h, rstd = B.rms_norm(x, w, residual=r)
        B.rms_norm_grad(dy, h, w, rstd)              # sizes the stream's workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, h, rstd = B.rms_norm(x, w, residual=r)
        dx, dw = B.rms_norm_grad(dy, h, w, rstd)
    for seed in (1, 2):
        nx, nr, _ = inputs(64, 2048, torch.bfloat16, torch.bfloat16, seed=10 * seed)
        x.copy_(nx)
        r.copy_(nr)
        graph.replay()
        torch.cuda.synchronize()
        y1, h1, rstd1 = B.rms_norm(nx, w, residual=nr)
        dx1, dw1 = B.rms_norm_grad(dy, h1, w, rstd1)
        for a, b in ((y, y1), (h, h1), (rstd, rstd1), (dx, dx1), (dw, dw1)):
            assert torch.equal(a, b)


def test_into_the_8_bit_product():
    """norm -> 8 bits -> product, against the product of the rounded values in 64 bits."""
    x, r, w = inputs(33, 640, torch.bfloat16, torch.float32)
    q, s, h = B.rms_norm_i8(x, w, residual=r)
    qw, sw = B.i8_quantize(rand(200, 640, seed=3, scale=0.04))
    y = B.i8_gemm(q, s, qw, sw, out_dtype=torch.float32)
    want = (q.double() @ qw.double().mT) * s.double()[:, None] * sw.double()
    close(y, want, want.abs() * 3 * U)
