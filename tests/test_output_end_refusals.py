"""Argument checks of the output end's calls: they return before any device call,
so they run without a GPU."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B
from dense_fp32_gemm_gb300 import layers

F32, BF16, F16 = B.SGEMM_TYPE_F32, B.SGEMM_TYPE_BF16, B.SGEMM_TYPE_F16
OK, VALUE, DIM, LD = B.SGEMM_OK, B.SGEMM_ERR_INVALID_VALUE, B.SGEMM_ERR_INVALID_DIM, B.SGEMM_ERR_INVALID_LD
NULL, ALIGN = B.SGEMM_ERR_NULL_PTR, B.SGEMM_ERR_MISALIGNED


NORM = dict(M=4, N=16, type=BF16, X=256, ldx=16, R=256, ldr=16, weight=256, weight_type=F32, eps=1e-6, H=256, ldh=16)
NORM_CASES = [
    (dict(type=3), VALUE), (dict(weight_type=F16), VALUE), (dict(weight_type=7), VALUE), (dict(eps=0.0), VALUE),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE), (dict(M=-1), DIM),
    (dict(N=-1), DIM), (dict(ldx=15), LD), (dict(ldr=15), LD), (dict(ldh=15), LD), (dict(X=None), NULL),
    (dict(weight=None), NULL), (dict(H=None), NULL), (dict(X=257), ALIGN), (dict(R=257), ALIGN), (dict(H=257), ALIGN),
    (dict(weight=258), ALIGN), (dict(M=0, X=None), OK), (dict(N=0, X=None), OK)]


@pytest.mark.parametrize("kw,want", NORM_CASES + [
    (dict(Y=None), NULL), (dict(Y=257), ALIGN), (dict(ldy=15), LD), (dict(rstd=258), ALIGN)])
def test_rms_norm(kw, want):
    assert B.sgemm_rms_norm(**(dict(NORM, Y=256, ldy=16, rstd=256) | kw)) == want


@pytest.mark.parametrize("kw,want", NORM_CASES + [
    (dict(Q=None), NULL), (dict(scale=None), NULL), (dict(scale=258), ALIGN), (dict(ldq=15), LD)])
def test_rms_norm_i8(kw, want):
    assert B.sgemm_rms_norm_i8(**(dict(NORM, Q=257, ldq=16, scale=256) | kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(type=3), VALUE), (dict(weight_type=F16), VALUE), (dict(M=-1), DIM), (dict(N=-1), DIM), (dict(lddy=15), LD),
    (dict(ldh=15), LD), (dict(lddh=15), LD), (dict(lddx=15), LD), (dict(dY=None), NULL), (dict(H=None), NULL),
    (dict(weight=None), NULL), (dict(rstd=None), NULL), (dict(dY=257), ALIGN), (dict(H=257), ALIGN),
    (dict(dH=257), ALIGN), (dict(dX=257), ALIGN), (dict(dweight=258), ALIGN), (dict(rstd=258), ALIGN),
    (dict(dX=None, dweight=None), OK), (dict(N=0, dY=None), OK)])
def test_rms_norm_grad(kw, want):
    a = dict(M=4, N=16, type=BF16, dY=256, lddy=16, H=256, ldh=16, weight=256, weight_type=F32, rstd=256, dH=256,
             lddh=16, dX=256, lddx=16, dweight=256)
    assert B.sgemm_rms_norm_grad(**(a | kw)) == want


def test_torch_norm_refuses():
    x, w, s = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    wide = torch.zeros(1, 8).expand(4, 8)
    for args, kw in [((x, w), {}),                                         # not on a GPU
                     ((x[0], w), {}), ((x.double(), w.double()), {}), ((x, w[:7]), {}), ((x, w.half()), {}),
                     ((x, torch.zeros(16)[::2]), {}), ((wide, w), {}), ((x.t(), s), {}), ((x, w), dict(residual=x[:3])),
                     ((x, w), dict(residual=x.half())), ((x, w), dict(residual=wide)), ((x, w), dict(H=x)),
                     ((x, w), dict(residual=x, H=x[:, :7]))]:
        for f in (B.rms_norm, B.rms_norm_i8):
            with pytest.raises(ValueError):
                f(*args, **kw)
    for kw in (dict(Y=x[:3]), dict(Y=x.half()), dict(Y=wide), dict(rstd=s[:3]), dict(rstd=s.double())):
        with pytest.raises(ValueError):
            B.rms_norm(x, w, **kw)
    for kw in (dict(Q=x), dict(scale=s[:3]), dict(Q=torch.zeros(4, 7, dtype=torch.int8))):
        with pytest.raises(ValueError):
            B.rms_norm_i8(x, w, **kw)
    for args, kw in [((x, x, w, s), {}), ((x[:3], x, w, s), {}), ((x.half(), x, w, s), {}), ((x, x, w, s[:3]), {}),
                     ((x, x, w[:7], s), {}), ((x, x, w, s), dict(dH=x[:3])), ((x, x, w, s), dict(dX=x.half())),
                     ((x, x, w, s), dict(dweight=w[:7])), ((wide, x, w, s), {})]:
        with pytest.raises(ValueError):
            B.rms_norm_grad(*args, **kw)
    with pytest.raises(ValueError):
        layers.rms_norm(x, w, residual=x[:3])
    with pytest.raises(TypeError):
        B.rms_norm(x, w, eps="small")


CE = dict(type=BF16, T=4, V=10, H=16, X=256, ldx=16, W=256, ldw=16, target=256, ignore_index=-100)
CE_CASES = [
    (dict(type=3), VALUE), (dict(T=-1), DIM), (dict(V=-1), DIM), (dict(H=-1), DIM), (dict(ldx=15), LD),
    (dict(ldw=15), LD), (dict(X=None), NULL), (dict(W=None), NULL), (dict(target=None), NULL), (dict(X=257), ALIGN),
    (dict(W=257), ALIGN), (dict(type=F32, X=258), ALIGN), (dict(target=260), ALIGN)]


@pytest.mark.parametrize("kw,want", CE_CASES + [
    (dict(loss=None), NULL), (dict(loss=258), ALIGN), (dict(lse=258), ALIGN), (dict(T=0, target=None), OK)])
def test_linear_ce(kw, want):
    assert B.sgemm_linear_ce(**(dict(CE, loss=256, lse=256) | kw)) == want


@pytest.mark.parametrize("kw,want", CE_CASES + [
    (dict(lse=None), NULL), (dict(dloss=None), NULL), (dict(lddx=15), LD), (dict(lddw=15), LD), (dict(lse=258), ALIGN),
    (dict(dloss=258), ALIGN), (dict(dX=257), ALIGN), (dict(dW=257), ALIGN), (dict(dX=None, dW=None), OK),
    (dict(H=0), OK)])
def test_linear_ce_grad(kw, want):
    a = dict(CE, lse=256, dloss=256, dX=256, lddx=16, dW=256, lddw=16)
    assert B.sgemm_linear_ce_grad(**(a | kw)) == want


def test_torch_loss_refuses():
    x, w, t, s = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    wide = torch.zeros(1, 8).expand(4, 8)
    for args, kw in [((x, w, t), {}),                                      # not on a GPU
                     ((x[0], w, t), {}), ((x, w[:, :7], t), {}), ((x, w.half(), t), {}), ((x.double(), w.double(), t), {}),
                     ((x, w, t[:3]), {}), ((x, w, t.int()), {}), ((x, w, t[:, None]), {}), ((wide, w, t), {}),
                     ((x, w.t(), t), {}), ((x, w, t), dict(loss=s[:3])), ((x, w, t), dict(lse=s.double()))]:
        with pytest.raises(ValueError):
            B.linear_cross_entropy(*args, **kw)
    for args, kw in [((x, w, t, s, s), {}), ((x, w, t, s[:3], s), {}), ((x, w, t, s, s.double()), {}),
                     ((x, w, t, s, s), dict(dX=w)), ((x, w, t, s, s), dict(dW=x)), ((x, w, t, s, s), dict(dX=wide))]:
        with pytest.raises(ValueError):
            B.linear_cross_entropy_grad(*args, **kw)
    with pytest.raises(TypeError):
        B.linear_cross_entropy(x, w, t, ignore_index=None)


@pytest.mark.parametrize("kw,want", [
    (dict(type=3), VALUE), (dict(M=-1), DIM), (dict(K=-1), DIM), (dict(ldx=39), LD), (dict(ldq=16), LD),
    (dict(ldq=40), LD), (dict(X=None), NULL), (dict(Q=None), NULL), (dict(scale=None), NULL), (dict(X=257), ALIGN),
    (dict(Q=264), ALIGN), (dict(scale=264), ALIGN), (dict(M=0, X=None), OK), (dict(K=0, X=None), OK)])
def test_mx4_quantize(kw, want):
    a = dict(M=4, K=40, type=BF16, X=256, ldx=40, Q=256, ldq=32, scale=256) | kw
    assert B.sgemm_mx4_quantize(**a) == want
    assert B.sgemm_mx4_dequantize(a["M"], a["K"], a["Q"], a["ldq"], a["scale"], a["type"], a["X"], a["ldx"]) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out_type=3), VALUE), (dict(M=-1), DIM), (dict(N=-1), DIM), (dict(K=-1), DIM), (dict(lda=16), LD),
    (dict(ldb=40), LD), (dict(ldc=7), LD), (dict(A=None), NULL), (dict(B=None), NULL), (dict(scaleA=None), NULL),
    (dict(scaleB=None), NULL), (dict(C=None), NULL), (dict(A=264), ALIGN), (dict(B=264), ALIGN),
    (dict(scaleA=264), ALIGN), (dict(scaleB=257), ALIGN), (dict(C=257), ALIGN), (dict(out_type=F32, C=258), ALIGN),
    (dict(M=0, A=None), OK), (dict(N=0, C=None), OK)])
def test_mx4(kw, want):
    a = dict(M=4, N=8, K=40, A=256, lda=32, scaleA=256, B=256, ldb=32, scaleB=256, out_type=BF16, C=256, ldc=8)
    assert B.sgemm_mx4(**(a | kw)) == want


def test_torch_mx4_refuses():
    x = torch.zeros(4, 40)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for args, kw in [((x,), {}), ((x[0],), {}), ((x.double(),), {}), ((x.t(),), {}), ((x,), dict(Q=q[:, :16])),
                     ((x,), dict(Q=q.to(torch.int8))), ((x,), dict(scale=s[:256])),
                     ((torch.zeros(1, 40).expand(4, 40),), {})]:
        with pytest.raises(ValueError):
            B.mx4_quantize(*args, **kw)
    odd = torch.zeros(4, 40, dtype=torch.uint8)[:, :32]
    for args, kw in [((q, s, 40), {}), ((q, s, 30), {}), ((q, s, 70), {}), ((q, s[:256], 40), {}), ((odd, s, 40), {}),
                     ((q, s, 40), dict(X=x[:3])), ((q, s, 40), dict(out_dtype=torch.float64))]:
        with pytest.raises(ValueError):
            B.mx4_dequantize(*args, **kw)
    for args, kw in [((q, s, q, s), {}), ((q[:, :16], s, q, s), {}), ((q, s[:256], q, s), {}), ((odd, s, q, s), {}),
                     ((q, s, q, s), dict(C=x)), ((q, s, q, s), dict(out_dtype=torch.int8)),
                     ((q.to(torch.int8), s, q, s), {})]:
        with pytest.raises(ValueError):
            B.mx4_gemm(*args, **kw)
    for bad in (s, x):
        with pytest.raises(ValueError):
            B.mx4_tile_scales(bad)
    t = B.mx4_tile_scales(torch.arange(200, dtype=torch.uint8).view(40, 5))
    assert t.shape == (1024,) and int(t[(33 % 32) * 16 + 4 + 2]) == 33 * 5 + 2 and int(t[512 + 7 * 16]) == 7 * 5 + 4
