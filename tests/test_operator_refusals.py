"""Argument checks of the grouped products, the 8-bit product and the gradient
clipping: they return before any device call, so they run without a GPU."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

T, N = B.SGEMM_OP_T, B.SGEMM_OP_N
F32, BF16, F16 = B.SGEMM_TYPE_F32, B.SGEMM_TYPE_BF16, B.SGEMM_TYPE_F16


def grouped(**kw):
    a = dict(op=T, type=BF16, out_type=BF16, E=2, T=8, N=16, K=24, alpha=1.0, X=256, ldx=24, W=256, ldw=24,
             strideW=384, offsets=256, beta=0.0, Y=256, ldy=16)
    a.update(kw)
    return B.sgemm_grouped(**a)


def wgrad(**kw):
    a = dict(type=BF16, out_type=F32, E=2, T=8, M=16, N=24, alpha=1.0, A=256, lda=16, B=256, ldb=24, offsets=256,
             beta=0.0, C=256, ldc=24, strideC=384)
    a.update(kw)
    return B.sgemm_grouped_wgrad(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(op=2), B.SGEMM_ERR_INVALID_VALUE), (dict(type=3), B.SGEMM_ERR_INVALID_VALUE),
    (dict(out_type=-1), B.SGEMM_ERR_INVALID_VALUE), (dict(type=F32), B.SGEMM_ERR_INVALID_VALUE),
    (dict(E=-1), B.SGEMM_ERR_INVALID_DIM), (dict(T=-1), B.SGEMM_ERR_INVALID_DIM),
    (dict(N=-1), B.SGEMM_ERR_INVALID_DIM), (dict(K=-1), B.SGEMM_ERR_INVALID_DIM),
    (dict(E=1025), B.SGEMM_ERR_INVALID_VALUE), (dict(strideW=-1), B.SGEMM_ERR_INVALID_VALUE),
    (dict(ldx=23), B.SGEMM_ERR_INVALID_LD), (dict(ldw=23), B.SGEMM_ERR_INVALID_LD),
    (dict(op=N, ldw=15), B.SGEMM_ERR_INVALID_LD), (dict(ldy=15), B.SGEMM_ERR_INVALID_LD),
    (dict(X=None), B.SGEMM_ERR_NULL_PTR), (dict(W=None), B.SGEMM_ERR_NULL_PTR),
    (dict(Y=None), B.SGEMM_ERR_NULL_PTR), (dict(offsets=None), B.SGEMM_ERR_NULL_PTR),
    (dict(X=257), B.SGEMM_ERR_MISALIGNED), (dict(Y=257), B.SGEMM_ERR_MISALIGNED),
    (dict(out_type=F32, Y=258), B.SGEMM_ERR_MISALIGNED), (dict(offsets=258), B.SGEMM_ERR_MISALIGNED),
    (dict(E=0, W=None, offsets=None), B.SGEMM_OK), (dict(T=0, X=None, Y=None), B.SGEMM_OK),
    (dict(N=0, Y=None), B.SGEMM_OK)])
def test_grouped(kw, want):
    assert grouped(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(type=9), B.SGEMM_ERR_INVALID_VALUE), (dict(type=F32, out_type=F16), B.SGEMM_ERR_INVALID_VALUE),
    (dict(M=-1), B.SGEMM_ERR_INVALID_DIM), (dict(T=-1), B.SGEMM_ERR_INVALID_DIM),
    (dict(E=5000), B.SGEMM_ERR_INVALID_VALUE), (dict(strideC=-1), B.SGEMM_ERR_INVALID_VALUE),
    (dict(lda=15), B.SGEMM_ERR_INVALID_LD), (dict(ldb=23), B.SGEMM_ERR_INVALID_LD),
    (dict(ldc=23), B.SGEMM_ERR_INVALID_LD), (dict(A=None), B.SGEMM_ERR_NULL_PTR),
    (dict(B=None), B.SGEMM_ERR_NULL_PTR), (dict(C=None), B.SGEMM_ERR_NULL_PTR),
    (dict(offsets=None), B.SGEMM_ERR_NULL_PTR), (dict(C=258), B.SGEMM_ERR_MISALIGNED),
    (dict(B=255), B.SGEMM_ERR_MISALIGNED), (dict(M=0, C=None), B.SGEMM_OK), (dict(E=0), B.SGEMM_OK)])
def test_wgrad(kw, want):
    assert wgrad(**kw) == want


def test_i8():
    def call(M=4, N=8, K=16, A=256, lda=16, sa=256, Bm=256, ldb=16, sb=256, out=F32, C=256, ldc=8):
        return B.sgemm_i8(M, N, K, A, lda, sa, Bm, ldb, sb, out, C, ldc)

    assert call(out=7) == B.SGEMM_ERR_INVALID_VALUE
    assert call(M=-1) == B.SGEMM_ERR_INVALID_DIM
    assert call(K=B.SGEMM_I8_MAX_K + 1, lda=1 << 20, ldb=1 << 20) == B.SGEMM_ERR_INVALID_DIM
    assert call(lda=15) == call(ldb=15) == call(ldc=7) == B.SGEMM_ERR_INVALID_LD
    assert call(A=None) == call(Bm=None) == call(sa=None) == call(sb=None) == call(C=None) == B.SGEMM_ERR_NULL_PTR
    assert call(C=258) == call(sa=257) == call(sb=258) == B.SGEMM_ERR_MISALIGNED
    assert call(M=0) == call(N=0) == B.SGEMM_OK


def test_i8_quantize():
    def call(M=4, K=16, t=BF16, X=256, ldx=16, Q=256, ldq=16, s=256):
        return B.sgemm_i8_quantize(M, K, t, X, ldx, Q, ldq, s)

    assert call(t=3) == B.SGEMM_ERR_INVALID_VALUE
    assert call(M=-1) == call(K=-2) == B.SGEMM_ERR_INVALID_DIM
    assert call(ldx=15) == call(ldq=15) == B.SGEMM_ERR_INVALID_LD
    assert call(X=None) == call(Q=None) == call(s=None) == B.SGEMM_ERR_NULL_PTR
    assert call(X=257) == call(t=F32, X=258) == call(s=258) == B.SGEMM_ERR_MISALIGNED
    assert call(M=0) == B.SGEMM_OK


def test_grad_clip():
    def call(grads=(256,), out=(256,), sizes=(4,), types=(F32,), most=1.0, norm=256):
        return B.sgemm_grad_clip(list(grads), None if out is None else list(out), list(sizes), list(types), most, norm)

    assert call(types=(5,)) == B.SGEMM_ERR_INVALID_VALUE
    assert call(most=-1.0) == call(most=float("nan")) == B.SGEMM_ERR_INVALID_VALUE
    assert call(sizes=(-1,)) == call(sizes=(1 << 41,)) == B.SGEMM_ERR_INVALID_DIM
    assert call(grads=(None,)) == call(out=(None,)) == call(out=None, norm=None) == B.SGEMM_ERR_NULL_PTR
    assert call(grads=(258,)) == call(out=(257,)) == call(norm=258) == B.SGEMM_ERR_MISALIGNED
    assert call(types=(F16,), grads=(257,)) == B.SGEMM_ERR_MISALIGNED


def test_torch_layer_refuses():
    x, w = torch.zeros(4, 8), torch.zeros(2, 6, 8)
    off = torch.zeros(3, dtype=torch.int32)
    for args, kw in [((x, w, off), {}),                                    # not on a GPU
                     ((x, w, off.long()), {}), ((x, w, off[:2]), {}), ((x, w, off), dict(op="C")),
                     ((x, w, off), dict(op="N")), ((x, w.half(), off), {}), ((x, w, off), dict(beta=1.0)),
                     ((x.double(), w.double(), off), {})]:
        with pytest.raises(ValueError):
            B.grouped_gemm(*args, **kw)
    for args in [(x, x, off), (x, x[:3], off), (x, x.half(), off), (x, x, off.float())]:
        with pytest.raises(ValueError):
            B.grouped_wgrad(*args)
    q = torch.zeros(4, 8, dtype=torch.int8)
    s = torch.zeros(4)
    for args in [(q, s, q, s), (x, s, q, s), (q, s[:3], q, s), (q, s, q[:, :7], s)]:
        with pytest.raises(ValueError):
            B.i8_gemm(*args)
    for args in [(x,), (x[0],)]:
        with pytest.raises(ValueError):
            B.i8_quantize(*args)
    for grads, kw in [([], {}), ([x], {}), ([x], dict(out=[])), ([x.t()], {})]:
        with pytest.raises(ValueError):
            B.clip_grad_norm(grads, 1.0, **kw)
