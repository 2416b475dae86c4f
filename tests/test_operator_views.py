"""Views whose rows overlap (expanded tensors, windows) have no row pitch: the
torch calls refuse them before any device call, so this runs without a GPU."""
import pytest
import torch

from dense_fp32_gemm_gb300 import binding as B

OVERLAP = "overlapping rows"
OFF = torch.zeros(3, dtype=torch.int32)


def mat(rows, cols, t=torch.float32):
    return torch.zeros(rows, cols, dtype=t)


def expanded(rows, cols, t=torch.float32):
    """One row `rows` times: strides (0, 1)."""
    return torch.zeros(cols, dtype=t).expand(rows, cols)


def windows(rows, cols, t=torch.float32):
    """Row i starts one element after row i - 1."""
    return torch.zeros(rows + cols, dtype=t).as_strided((rows, cols), (1, 1))


@pytest.mark.parametrize("view", [expanded, windows])
def test_grouped_gemm(view):
    w = torch.zeros(2, 6, 8)
    for x, w3, y in [(view(4, 8), w, None), (mat(4, 8), view(6, 8).expand(2, 6, 8), None), (mat(4, 8), w, view(4, 6))]:
        with pytest.raises(ValueError, match=OVERLAP):
            B.grouped_gemm(x, w3, OFF, Y=y)


def test_one_column_repeated():
    with pytest.raises(ValueError, match=OVERLAP):
        B.grouped_gemm(torch.zeros(1, 1).expand(4, 1), torch.zeros(2, 6, 1), OFF)


@pytest.mark.parametrize("view", [expanded, windows])
def test_grouped_wgrad(view):
    for a, b, c in [(view(4, 8), mat(4, 6), None), (mat(4, 8), view(4, 6), None),
                    (mat(4, 8), mat(4, 6), view(8, 6).expand(2, 8, 6))]:
        with pytest.raises(ValueError, match=OVERLAP):
            B.grouped_wgrad(a, b, OFF, C=c)


@pytest.mark.parametrize("view", [expanded, windows])
def test_i8(view):
    i8 = torch.int8
    with pytest.raises(ValueError, match=OVERLAP):
        B.i8_quantize(view(4, 8))
    with pytest.raises(ValueError, match=OVERLAP):
        B.i8_quantize(mat(4, 8), Q=view(4, 8, i8), scale=torch.zeros(4))
    s4, s5 = torch.zeros(4), torch.zeros(5)
    for a, b, c in [(view(4, 8, i8), mat(5, 8, i8), None), (mat(4, 8, i8), view(5, 8, i8), None),
                    (mat(4, 8, i8), mat(5, 8, i8), view(4, 5))]:
        with pytest.raises(ValueError, match=OVERLAP):
            B.i8_gemm(a, s4, b, s5, C=c)


@pytest.mark.parametrize("view", [expanded, windows])
def test_gemm_leading_dimension(view):
    with pytest.raises(ValueError, match=OVERLAP):
        B._ld(view(4, 8), "A")


def test_views_that_do_not_overlap_keep_their_pitch():
    assert B._ld(mat(4, 8), "A") == 8 and B._ld(mat(4, 8)[:, :5], "A") == 8
    assert B._ld(mat(4, 8)[::2], "A") == 16 and B._ld(mat(1, 8).expand(1, 8), "A") == 8
    assert B._ld(mat(4, 1), "A") == 1 and B._ld(mat(0, 8), "A") == 8 and B._ld(mat(1, 0).expand(4, 0), "A") == 1
    # on the CPU what is left to refuse is the device
    for x in (mat(4, 8), mat(8, 16)[::2, 3:11], mat(1, 8).expand(1, 8)):
        with pytest.raises(ValueError, match="CUDA device"):
            B.grouped_gemm(x, torch.zeros(2, 6, 8), OFF)


def negated(*shape):
    """A view whose values are the stored ones with the other sign, one column of each row."""
    z = torch.ones(*shape, 2, dtype=torch.complex64)
    return z.conj().imag[..., :1]


def test_negated_views():
    """What the kernels would read of them has the wrong sign."""
    x, w, n1 = mat(4, 1), torch.zeros(2, 1, 1), negated(4)
    assert n1.is_neg() and n1.shape == (4, 1)
    for call in (lambda: B.grouped_gemm(n1, w, OFF), lambda: B.grouped_gemm(x, negated(2, 1), OFF),
                 lambda: B.grouped_gemm(x, w, OFF, Y=n1), lambda: B.grouped_wgrad(n1, x, OFF),
                 lambda: B.grouped_wgrad(x, n1, OFF), lambda: B.grouped_wgrad(x, x, OFF, C=negated(2, 1)),
                 lambda: B.i8_quantize(n1), lambda: B._ld(n1, "A"),
                 lambda: B.i8_gemm(x.to(torch.int8), torch.zeros(4), mat(1, 1, torch.int8), torch.zeros(1), C=n1)):
        with pytest.raises(ValueError, match="negated view"):
            call()


def test_wgrad_groups_that_share_elements():
    a, b = mat(4, 8), mat(4, 6)
    for c in (mat(8, 6).expand(2, 8, 6), torch.zeros(100).as_strided((2, 8, 6), (47, 6, 1)),
              torch.zeros(200).as_strided((2, 8, 6), (5, 12, 1)), torch.zeros(200).as_strided((2, 8, 6), (6, 11, 1))):
        with pytest.raises(ValueError, match="matrices in C overlap"):
            B.grouped_wgrad(a, b, OFF, C=c)
    # one after another, and row by row beside each other
    for c in (torch.zeros(2, 8, 6), torch.zeros(8, 2, 6).transpose(0, 1), torch.zeros(2, 9, 7)[:, 1:, :6],
              torch.zeros(1, 8, 6).expand(2, 8, 6)[:1]):
        off = OFF if c.size(0) == 2 else OFF[:2]
        with pytest.raises(ValueError, match="CUDA device"):
            B.grouped_wgrad(a, b, off, C=c)
