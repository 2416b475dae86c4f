"""Rows at the borders between the ways in which they are taken (16-byte pieces some
lanes a row, shifted pieces, single elements of one warp), many to a call, against the
64-bit formulas with the tolerances of the norm's own tests (a row here has at most
257 values, on 32 threads: 9 additions one after another and a tree of 5)."""
import pytest
import torch

import test_gpu_rms_norm as norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [125, 126, 129, 189, 197, 249, 250, 253, 254, 255, 257])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
def test_many_rows(t, n):
    for m in (303, 1234):           # below and above two rows a multiprocessor
        norm.test_forward(t, m, n, True)
        norm.test_8_bits(t, m, n)
        norm.test_gradients(t, m, n, True)
