"""Calls of the 4-bit operators that the documentation allows and that are easy
to get wrong: slices of one buffer, tensors without features, factors, seeds,
gradients beside autograd."""
import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from oracle import mx_oracle as mx
from tests.gpu_helpers import announce, host

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def _rand(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(dtype).cuda()


def test_outputs_that_are_slices_of_one_buffer():
    """A single row, a column slice and every second row of one buffer share nothing."""
    announce("one buffer's slices as outputs")
    xs = [mo.mx_quantize(_rand(r, 64, BF16, r)) for r in (1, 17, 9)]
    w = mo.mx_quantize(_rand(30, 64, BF16, 40))
    buf = torch.full((18, 100), 7.0, device="cuda")
    outs = [buf[1:2, :30], buf[:17, 30:60], buf[::2, 60:90]]
    mo.mx_matmul(xs, [w] * 3, out=outs)
    for o, x in zip(outs, xs):
        assert torch.equal(o, mo.mx_matmul(x, w, dtype=F32))
    assert bool((buf[0, :30] == 7.0).all() and (buf[2:, :30] == 7.0).all() and (buf[1::2, 60:] == 7.0).all())
    with pytest.raises(mo._lib.MuonError):
        mo.mx_matmul(xs, [w] * 3, out=[buf[1:2, 1:31], buf[:17, 30:60], buf[::2, 60:90]])
    x = _rand(17, 60, BF16, 3)
    wide = torch.zeros(17, 120, dtype=BF16, device="cuda")
    wide[:, :60] = x
    mo.dropout(wide[4:5, :60], 0.3, 9, out=wide[4:5, 60:])
    assert torch.equal(wide[4:5, 60:], mo.dropout(x[4:5], 0.3, 9)) and torch.equal(wide[:, :60], x)
