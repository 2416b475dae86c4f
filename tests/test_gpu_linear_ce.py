"""Softmax cross entropy over a vocabulary and its gradients, against the formulas
in 64 bits.

Tolerances. A logit is a sum of exact products in FP32 (or of products off by
2^-23) that leaves the tensor cores, which truncate, after at most 64
instructions: it is off by at most 64 * 2^-23 < 8e-6 of the sum of magnitudes S.
lse moves by no more than its logits do; its exponentials are off by 2^-22 and
what |z - max| 2^-23 gives, weighted by themselves, 1e-6 in all. The loss, of two
logits, by 16e-6 S. G is rounded to the operands' type (half a unit) and its
probabilities carry the errors of two logits; the products truncate again."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from dense_fp32_gemm_gb300 import layers

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
IGNORE = -100
U = 2.0 ** -24


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def rounding(want, t):
    """Half a step of type t at the values `want`."""
    f = torch.finfo(t)
    return torch.maximum(want.abs() * f.eps / 2, torch.full_like(want, f.smallest_normal * f.eps / 2))


def inputs(t, v, h, dtype, seed=0, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    target[torch.rand((t,), generator=g, device="cuda") < ignored] = IGNORE
    return rand(t, h, seed=seed).to(dtype), rand(v, h, seed=seed + 1, scale=2 * h ** -0.5).to(dtype), target


def formula(x, w, target, d=None):
    """loss, lse, S (largest sum of magnitudes of a row's logits); with d also P and G."""
    x, w = x.double(), w.double()
    z = x @ w.mT
    lse = torch.logsumexp(z, dim=1)
    counted = target != IGNORE
    at = torch.where(counted, target, 0)[:, None]
    loss = torch.where(counted, lse - z.gather(1, at)[:, 0], 0.0)
    s = (x.abs() @ w.abs().mT).amax(dim=1)
    if d is None:
        return loss, lse, s
    p = (z - lse[:, None]).exp()
    g = p.clone()
    g.scatter_add_(1, at, torch.full_like(lse[:, None], -1.0))
    d = torch.where(counted, d.double(), 0.0)[:, None]
    return loss, lse, s, p * d.abs(), g * d


def close(got, want, slack, what=""):
    off = (got.double() - want).abs() - slack
    assert bool((off <= 0).all()), f"{what} off by {float(off.max()):.3g} more than allowed"


def check(x, w, target, d, loss, lse, dx, dw):
    dtype = x.dtype
    ref_loss, ref_lse, s, p, g = formula(x, w, target, d)
    close(lse, ref_lse, 8e-6 * s + 2e-6 + ref_lse.abs() * 2 * U, "lse")
    close(loss, ref_loss, 16e-6 * s + 2e-6 + ref_lse.abs() * 4 * U, "loss")
    unit = torch.finfo(dtype).eps / 2
    # (F16: below 2^-14 of the largest |d| / 2^14 steps no longer shrink)
    least = float(d.abs().amax()) * 2.0 ** -38 if dtype == torch.float16 and d.numel() else 0.0
    off_g = unit * g.abs() + (16e-6 * s + 3e-6)[:, None] * p + least
    xd, wd = x.double().abs(), w.double().abs()
    if dx is not None:
        want = g @ w.double()
        close(dx, want, off_g @ wd + 1e-5 * (g.abs() @ wd) + rounding(want, dtype), "dx")
    if dw is not None:
        want = g.mT @ x.double()
        close(dw, want, off_g.mT @ xd + 1e-5 * (g.abs().mT @ xd) + rounding(want, dtype), "dw")


SIZES = [(1, 1, 1), (1, 1000, 64), (7, 33, 5), (65, 1000, 256), (130, 777, 100), (300, 5000, 520), (257, 1023, 1030),
         (1000, 300, 2048), (2, 70001, 72), (513, 2, 8)]


@pytest.mark.parametrize("t,v,h", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_and_gradients(dtype, t, v, h):
    x, w, target = inputs(t, v, h, dtype)
    d = rand(t, seed=9)
    loss, lse = B.linear_cross_entropy(x, w, target)
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    assert dx.dtype == dw.dtype == dtype and loss.dtype == lse.dtype == torch.float32
    check(x, w, target, d, loss, lse, dx, dw)
    assert not bool(loss[target == IGNORE].any()) and not bool(dx[target == IGNORE].any())
    # one of the two gradients alone is the same
    only_x, none = B.linear_cross_entropy_grad(x, w, target, lse, d, want=(True, False))
    also_none, only_w = B.linear_cross_entropy_grad(x, w, target, lse, d, want=(False, True))
    assert none is None and also_none is None and torch.equal(only_x, dx) and torch.equal(only_w, dw)


@pytest.mark.parametrize("dtype", TYPES)
def test_exact_logits(dtype):
    """Small integers: the logits are exact, so only the exponentials and their sum are off."""
    t, v, h = 200, 3000, 96
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-1, 2, (t, h), generator=g, device="cuda").to(dtype)
    w = torch.randint(-1, 2, (v, h), generator=g, device="cuda").to(dtype)
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    loss, lse = B.linear_cross_entropy(x, w, target)
    ref_loss, ref_lse, _ = formula(x, w, target)
    close(lse, ref_lse, 2e-6 + ref_lse.abs() * 2 * U)
    close(loss, ref_loss, 2e-6 + ref_lse.abs() * 4 * U)


@pytest.mark.parametrize("tile", [(64, 1), (128, 1), (256, 1), (256, 2), (16, 1)])
def test_every_tile(tile):
    """Every built form, with tiles that are cut along h and with whole ones."""
    for t, v, h, dtype in ((300, 900, 4000, torch.bfloat16), (5000, 3000, 72, torch.float16)):
        x, w, target = inputs(t, v, h, dtype)
        d = rand(t, seed=9)
        try:
            assert B.sgemm_grouped_set_tile(*tile) == 0
            loss, lse = B.linear_cross_entropy(x, w, target)
            if tile[0] >= 64:
                assert f"x{tile[0]}x" in B.sgemm_last_config()
            dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
        finally:
            B.sgemm_grouped_set_tile(0)
        check(x, w, target, d, loss, lse, dx, dw)


@pytest.mark.parametrize("tile", [(16, 1), (32, 1), (64, 1)])
def test_few_tokens(tile):
    """Words on the lanes: every built form, words and tokens that end inside a tile, tiles cut along h."""
    for t, v, h, dtype in ((1, 70, 3000, torch.bfloat16), (40, 1000, 4000, torch.float16), (64, 20001, 72, torch.bfloat16),
                           (17, 129, 8, torch.float16)):
        x, w, target = inputs(t, v, h, dtype)
        target[0], target[-1] = v - 1, 0
        d = rand(t, seed=9)
        try:
            assert B.sgemm_grouped_set_tile(*tile) == 0
            loss, lse = B.linear_cross_entropy(x, w, target)
            assert f"128x{tile[0]}x" in B.sgemm_last_config()
            dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
        finally:
            B.sgemm_grouped_set_tile(0)
        check(x, w, target, d, loss, lse, dx, dw)


@pytest.mark.parametrize("dtype", TYPES)
def test_several_pieces(dtype):
    """G (or FP32 logits) of more than the workspace's share."""
    t, v, h = (8200, 40000, 40) if dtype != torch.float32 else (4100, 40000, 40)
    x, w, target = inputs(t, v, h, dtype)
    target[:8] = torch.tensor([0, v - 1, v // 2, v // 2 - 1, 20223, 20224, 19999, 20000], device="cuda")
    d = rand(t, seed=9)
    loss, lse = B.linear_cross_entropy(x, w, target)
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    check(x, w, target, d, loss, lse, dx, dw)


@pytest.mark.parametrize("t,v", [(66000, 18000), (600001, 2500)])
def test_several_pieces_of_the_loss(t, v):
    x, w, target = inputs(t, v, 16, torch.bfloat16)
    loss, lse = B.linear_cross_entropy(x, w, target)
    for a in range(0, t, 50000):
        r = slice(a, a + 50000)
        ref_loss, ref_lse, s = formula(x[r], w, target[r])
        close(lse[r], ref_lse, 8e-6 * s + 2e-6 + ref_lse.abs() * 2 * U)
        close(loss[r], ref_loss, 16e-6 * s + 2e-6 + ref_lse.abs() * 4 * U)


@pytest.mark.parametrize("dtype", TYPES)
def test_targets_that_are_none(dtype):
    x, w, target = inputs(70, 500, 64, dtype, ignored=0.0)
    target[3], target[4], target[5] = 500, -1, 1 << 40
    d = torch.ones(70, device="cuda")
    loss, lse = B.linear_cross_entropy(x, w, target)
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[3:6] = True
    assert torch.equal(loss.isnan(), bad) and not bool(lse.isnan().any())
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    assert bool(dx[bad].isnan().all()) and not bool(dx[~bad].isnan().any()) and bool(dw.isnan().all())
    # another ignore_index, a word among them
    target[3:6] = 17
    loss, lse = B.linear_cross_entropy(x, w, target, ignore_index=17)
    assert not bool(loss[target == 17].any())
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d, ignore_index=17)
    again = torch.where(target == 17, IGNORE, target)
    check(x, w, again, d, loss, lse, dx, dw)
    # no row counts
    target[:] = IGNORE
    loss, lse = B.linear_cross_entropy(x, w, target)
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("dtype", TYPES)
def test_no_numbers(dtype):
    x, w, target = inputs(40, 600, 64, dtype, ignored=0.0)
    target[7] = IGNORE
    clean = B.linear_cross_entropy(x, w, target)[0]
    x[5, 3], x[7, 0] = float("nan"), float("nan")
    loss, _ = B.linear_cross_entropy(x, w, target)
    assert bool(loss[5].isnan()) and float(loss[7]) == 0.0
    keep = [i for i in range(40) if i != 5]
    assert torch.equal(loss[keep], clean[keep])
    # a word that can never come: its logits are -infinity
    x, w, target = inputs(40, 600, 64, dtype, ignored=0.0)
    x = x.abs()
    if dtype != torch.float32:      # (an infinite FP32 operand gives NaN)
        target[target == 599] = 0
        w[599] = float("-inf")
        loss, lse = B.linear_cross_entropy(x, w, target)
        ref = torch.logsumexp(x.double() @ w[:599].double().mT, dim=1)
        s = (x.double() @ w[:599].double().abs().mT).amax(dim=1)
        close(lse, ref, 8e-6 * s + 2e-6 + ref.abs() * 2 * U)
        w[598] = float("inf")
        assert bool(B.linear_cross_entropy(x, w, target)[0].isnan().all())


def test_large_logits():
    """Logits of some 10^4: no exponential overflows, and the largest word has nearly all of the probability."""
    x, w, target = inputs(64, 1000, 128, torch.bfloat16, ignored=0.0)
    x, w = (x * 64), (w * 64)
    d = torch.ones(64, device="cuda")
    loss, lse = B.linear_cross_entropy(x, w, target)
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
    ref_loss, ref_lse, s = formula(x, w, target)
    close(lse, ref_lse, 8e-6 * s + 2e-6 + ref_lse.abs() * 2 * U)
    close(loss, ref_loss, 16e-6 * s + 2e-6 + ref_lse.abs() * 4 * U)
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
def test_upstream_gradients(dtype):
    """Tiny, zero, infinite and NaN gradients of the losses."""
    x, w, target = inputs(90, 400, 64, dtype, ignored=0.1)
    loss, lse = B.linear_cross_entropy(x, w, target)
    d = rand(90, seed=4, scale=1e-3)
    check(x, w, target, d, loss, lse, *B.linear_cross_entropy_grad(x, w, target, lse, d))
    zero = torch.zeros(90, device="cuda")
    dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, zero)
    assert not bool(dx.any()) and not bool(dw.any())
    row = int((target != IGNORE).nonzero()[0])
    for bad in (float("nan"), float("inf")):
        e = d.clone()
        e[row] = bad
        dx, _ = B.linear_cross_entropy_grad(x, w, target, lse, e)
        wrong = ~dx.isfinite().all(dim=1)
        assert bool(wrong[row]) and int(wrong.sum()) == 1
    # what stands beside a row that is not counted is not looked at
    e = d.clone()
    e[target == IGNORE] = float("nan")
    a, b = B.linear_cross_entropy_grad(x, w, target, lse, e), B.linear_cross_entropy_grad(x, w, target, lse, d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("size", [1e3, 1e-9])
@pytest.mark.parametrize("dtype", TYPES)
def test_an_infinite_upstream_gradient_leaves_the_other_rows(dtype, size):
    """Rows of dX do not depend on another row's dloss, but for the largest number
    among them, which G is scaled by."""
    x, w, target = inputs(90, 400, 64, dtype, ignored=0.1)
    _, lse = B.linear_cross_entropy(x, w, target)
    counted = (target != IGNORE).nonzero()
    row = int(counted[0])
    d = rand(90, seed=4, scale=size)
    d[int(counted[1])] = 8 * size                        # the largest, without `row` and with it
    d[row] = 0
    want = B.linear_cross_entropy_grad(x, w, target, lse, d)[0]
    assert bool(want.isfinite().all())
    d[row] = float("inf")
    got = B.linear_cross_entropy_grad(x, w, target, lse, d)[0]
    others = torch.arange(90, device="cuda") != row
    assert torch.equal(got[others], want[others]) and not bool(got[row].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3)])
def test_strides_and_guards(dtype, offset, pad):
    t, v, h = 150, 700, 88
    x, w, target = inputs(t, v, h, dtype)
    d = rand(t, seed=9)

    def buffer(rows, values=None):
        store = torch.full((offset + rows * (h + pad) + 16,), 77, dtype=dtype, device="cuda")
        view = store[offset: offset + rows * (h + pad)].view(rows, h + pad)[:, :h]
        if values is not None:
            view.copy_(values)
        return store, view

    (_, xv), (_, wv), (dxs, dxv), (dws, dwv) = buffer(t, x), buffer(v, w), buffer(t), buffer(v)
    rows = torch.full((t + 2,), 77.0, device="cuda")
    loss, lse = B.linear_cross_entropy(xv, wv, target, loss=rows[1:-1])
    assert float(rows[0]) == float(rows[-1]) == 77.0
    dx, dw = B.linear_cross_entropy_grad(xv, wv, target, lse, d, dX=dxv, dW=dwv)
    assert dx is dxv and dw is dwv
    check(x, w, target, d, loss, lse, dx, dw)
    for store, rows in ((dxs, t), (dws, v)):
        mask = torch.ones(store.numel(), dtype=torch.bool, device="cuda")
        mask[offset: offset + rows * (h + pad)].view(rows, h + pad)[:, :h] = False
        assert bool((store[mask] == 77).all())


def test_empty():
    for dtype in TYPES:
        x, w = torch.zeros(0, 16, dtype=dtype, device="cuda"), rand(50, 16).to(dtype)
        target = torch.zeros(0, dtype=torch.int64, device="cuda")
        loss, lse = B.linear_cross_entropy(x, w, target)
        dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, loss)
        assert loss.shape == (0,) and dx.shape == (0, 16) and not bool(dw.any())
        # no features: all logits are 0
        x, w = torch.zeros(5, 0, dtype=dtype, device="cuda"), torch.zeros(50, 0, dtype=dtype, device="cuda")
        loss, lse = B.linear_cross_entropy(x, w, torch.arange(5, device="cuda"))
        close(loss, torch.full((5,), 50.0, device="cuda").double().log(), 1e-6)
        # no words: nothing can be counted
        x, w = rand(5, 16).to(dtype), torch.zeros(0, 16, dtype=dtype, device="cuda")
        target = torch.full((5,), IGNORE, device="cuda")
        loss, lse = B.linear_cross_entropy(x, w, target)
        dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, loss)
        assert not bool(loss.any()) and not bool(dx.any()) and dw.shape == (0, 16)


def test_gradient_against_differences():
    t, v, h = 20, 130, 48
    x, w, target = inputs(t, v, h, torch.float32)
    leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    layers.linear_cross_entropy(leaves[0], leaves[1], target).backward()
    step = 1e-5

    def mean(x, w):
        return formula(x, w, target)[0].sum() / (target != IGNORE).sum()

    for i, leaf in enumerate(leaves):
        u = rand(*leaf.shape, seed=30 + i).double()
        at = [x.double(), w.double()]
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + step * u, at[i] - step * u
        slope = (mean(*plus) - mean(*minus)) / (2 * step)
        got = (leaf.grad.double() * u).sum()
        # the quotient: step^2 times a third derivative of some 10; the gradients as in check(), some 2e-5
        size = (leaf.grad.double() * u).abs().sum()
        assert abs(float(slope - got)) <= 1e-8 + 3e-5 * float(size)


def test_reductions():
    x, w, target = inputs(24, 90, 32, torch.float32)
    x3, t3 = x.view(4, 6, 32), target.view(4, 6)
    rows = layers.linear_cross_entropy(x3, w, t3, reduction="none")
    assert rows.shape == (4, 6)
    assert torch.equal(layers.linear_cross_entropy(x3, w, t3, reduction="sum"), rows.view(-1).sum())
    count = int((target != IGNORE).sum())
    assert abs(float(layers.linear_cross_entropy(x3, w, t3)) - float(rows.sum()) / count) < 1e-6
    wr = w.clone().requires_grad_()
    layers.linear_cross_entropy(x3, wr, torch.full_like(t3, IGNORE)).backward()
    assert not bool(wr.grad.any())
    with pytest.raises(ValueError):
        layers.linear_cross_entropy(x3, w, target)
    with pytest.raises(ValueError):
        layers.linear_cross_entropy(x3, w, t3, reduction="most")


def test_same_bits_each_time_and_on_another_stream():
    x, w, target = inputs(700, 9000, 512, torch.bfloat16)
    d = rand(700, seed=9)

    def all_of(stream=None):
        loss, lse = B.linear_cross_entropy(x, w, target, stream=stream)
        return (loss, lse) + B.linear_cross_entropy_grad(x, w, target, lse, d, stream=stream)

    first = all_of()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    second = all_of(other)
    torch.cuda.current_stream().wait_stream(other)
    for a, b, c in zip(first, second, all_of()):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured(dtype):
    x, w, target = inputs(200, 3000, 256, dtype)
    d = rand(200, seed=9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        loss, lse = B.linear_cross_entropy(x, w, target)
        B.linear_cross_entropy_grad(x, w, target, lse, d)          # sizes the stream's workspace
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                             # two graphs that share it
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loss, lse = B.linear_cross_entropy(x, w, target)
            dx, dw = B.linear_cross_entropy_grad(x, w, target, lse, d)
        graphs.append((graph, loss, lse, dx, dw))
    for seed in (1, 2):
        nx, nw, nt = inputs(200, 3000, 256, dtype, seed=10 * seed)
        x.copy_(nx)
        w.copy_(nw)
        target.copy_(nt)
        for graph, *out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        loss, lse = B.linear_cross_entropy(nx, nw, nt)
        want = (loss, lse) + B.linear_cross_entropy_grad(nx, nw, nt, lse, d)
        for _, *out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_capture_needs_the_workspace():
    x, w, target = inputs(64, 500, 64, torch.bfloat16)
    torch.cuda.synchronize()
    B.sgemm_shutdown()                                   # no stream has one (torch hands out streams again)
    want = B.linear_cross_entropy(x, w, target)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(B.SgemmError) as e:
        with torch.cuda.graph(graph, stream=side):
            B.linear_cross_entropy(x, w, target)
    assert e.value.status == B.SGEMM_ERR_CAPTURE
    torch.cuda.synchronize()
    assert torch.equal(B.linear_cross_entropy(x, w, target, stream=side)[0], want)


def test_norm_loss_and_clipping():
    """A training step's end: norm, loss, backward through both, clipping; against autograd in 64 bits."""
    t, v, h = 96, 700, 128
    x, w, target = inputs(t, v, h, torch.float32)
    r, g = rand(t, h, seed=11), 1 + 0.1 * rand(h, seed=12)
    leaves = [a.clone().requires_grad_() for a in (x, r, g, w)]
    y, _ = layers.rms_norm(leaves[0], leaves[2], residual=leaves[1])
    loss = layers.linear_cross_entropy(y, leaves[3], target)
    grads = list(torch.autograd.grad(loss, leaves))
    wide = [a.double().requires_grad_() for a in (x, r, g, w)]
    hsum = wide[0] + wide[1]
    n = hsum / (hsum.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * wide[2]
    ref_loss = formula(n, wide[3], target)[0].sum() / (target != IGNORE).sum()
    ref = torch.autograd.grad(ref_loss, wide)
    assert abs(loss.item() - ref_loss.item()) < 1e-4 * ref_loss.item()
    for a, b in zip(grads, ref):
        assert float((a.double() - b).norm()) <= 5e-5 * float(b.norm())
    norm = B.clip_grad_norm(grads, 0.1)
    want = torch.sqrt(sum(b.square().sum() for b in ref))
    assert abs(float(norm) - float(want)) <= 1e-4 * float(want)
