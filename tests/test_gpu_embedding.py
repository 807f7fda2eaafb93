"""The embedding table's lookup and gradient on the GPU against the float64 oracle.

A lookup is one fp32 product and one rounding to the table's type.  A gradient's
entry is an fp32 sum of n terms in some order, n 2^-23 of their magnitudes' sum
at most however additions round, a product with the scale and a rounding to its
type."""
import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from oracle import sparse_oracle as so
from tests.gpu_helpers import announce, host

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def half(dtype):
    return 2.0 ** -8 if dtype == BF16 else U


def ids_of(g, tokens, rows, kind):
    if kind == "same":
        return torch.full((tokens,), rows // 2)
    if kind == "spread":
        return torch.randint(0, rows, (tokens,), generator=g)
    u = torch.rand(tokens, generator=g).double()               # a few ids far more often than the rest
    ids = (torch.exp(u * np.log(rows + 1)).long().clamp(1, rows) - 1)
    if kind == "padded":
        ids[torch.rand(tokens, generator=g) < 0.3] = -1
        ids[torch.rand(tokens, generator=g) < 0.05] = rows
        ids[torch.rand(tokens, generator=g) < 0.05] = rows + 2 ** 33
    return ids


@pytest.mark.parametrize("kind", ["words", "same", "spread", "padded"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 1, 1), (5, 3, 8), (33, 300, 77), (64, 70000, 24), (1000, 50, 33), (256, 700, 1030), (257, 40, 8),
                                              (1025, 5000, 520), (2500, 70, 1030), (33000, 40, 9)])
def test_lookup_and_gradient(tokens, rows, cols, dtype, kind):
    announce(f"embedding {tokens} of {rows} x {cols}, {dtype}, {kind}")
    g = torch.Generator().manual_seed(tokens + rows)
    ids = ids_of(g, tokens, rows, kind)
    w, dy = torch.randn(rows, cols, generator=g).to(dtype), torch.randn(tokens, cols, generator=g).to(dtype)
    scale = 0.7
    s32 = float(np.float32(scale))
    wh, dh = w.double().numpy(), dy.double().numpy()
    got = host(mo.embedding(ids.cuda(), w.cuda(), scale)).astype(np.float64)
    want = so.embedding(ids.numpy(), wh, s32)
    assert (np.abs(got - want) <= (U + half(dtype)) * np.abs(want) * (1 + U)).all()
    assert torch.equal(mo.embedding(ids.cuda(), w.cuda()).cpu(), torch.where(
        ((ids >= 0) & (ids < rows)).unsqueeze(1), w[ids.clamp(0, rows - 1)], torch.zeros((), dtype=dtype)))
    dw = mo.embedding_grad(dy.cuda(), ids.cuda(), rows, scale)
    want, s = so.embedding_grad(dh, ids.numpy(), rows, s32), so.embedding_grad(np.abs(dh), ids.numpy(), rows, s32)
    count = np.bincount(ids.numpy()[(ids.numpy() >= 0) & (ids.numpy() < rows)], minlength=rows)[:, None]
    tol = (count + 1) * 2 * U * s
    assert dw.dtype == F32 and (np.abs(host(dw) - want) <= tol + U * np.abs(want)).all()
    # the same bits again, from int32 ids, in another type and added
    if kind != "padded":
        assert torch.equal(mo.embedding_grad(dy.cuda(), ids.int().cuda(), rows, scale), dw)
    assert torch.equal(mo.embedding_grad(dy.cuda(), ids.cuda(), rows, scale, grad_dtype=BF16), dw.to(BF16))
    old = torch.randn(rows, cols, generator=g).cuda()
    out = old.clone()
    assert mo.embedding_grad(dy.cuda(), ids.cuda(), rows, scale, out=out, accumulate=True) is out
    tol = tol + 2 * U * (np.abs(want) + np.abs(host(old)))
    assert (np.abs(host(out) - (want + host(old).astype(np.float64))) <= tol).all()
    assert torch.equal(out[torch.from_numpy(count[:, 0] == 0).cuda()], old[torch.from_numpy(count[:, 0] == 0).cuda()])


@pytest.mark.parametrize("rows", [200, 300, 70000, 2000000])
def test_long_sorts(rows):
    """Tokens in one block, in few and in many, keys of one to three digits: exact sums of small integers."""
    g = torch.Generator().manual_seed(rows)
    for tokens in (1024, 32768, 40000, (1 << 20) + 77):
        announce(f"sort {tokens} of {rows}")
        ids = ids_of(g, tokens, rows, "words")
        dy = torch.randint(-8, 9, (tokens, 3), generator=g).float()
        got = mo.embedding_grad(dy.cuda(), ids.cuda(), rows)
        want = torch.zeros(rows, 3).index_add_(0, ids, dy)
        assert torch.equal(got.cpu(), want)


def test_shapes_strides_and_empty_calls():
    g = torch.Generator().manual_seed(3)
    w, ids = torch.randn(50, 40, generator=g).cuda(), torch.randint(0, 50, (3, 7), generator=g).cuda()
    y = mo.embedding(ids, w)
    assert y.shape == (3, 7, 40) and torch.equal(y, w[ids])
    assert torch.equal(mo.embedding(ids, w[:, 3:24]), w[:, 3:24][ids])
    room = torch.zeros(3, 7, 48, device="cuda")
    mo.embedding(ids, w, out=room[:, :, 5:45])
    assert torch.equal(room[:, :, 5:45], w[ids]) and not room[:, :, :5].any() and not room[:, :, 45:].any()
    dy = torch.randn(3, 7, 48, generator=g).cuda()
    a = mo.embedding_grad(dy[:, :, 3:43], ids, 50)
    b = mo.embedding_grad(dy[:, :, 3:43].contiguous(), ids, 50)
    assert torch.equal(a, b)
    out = torch.full((50, 48), 2.0, device="cuda")
    mo.embedding_grad(dy[:, :, 3:43], ids, 50, out=out[:, 4:44])
    assert torch.equal(out[:, 4:44], a) and (out[:, :4] == 2).all() and (out[:, 44:] == 2).all()
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert mo.embedding(none, w).shape == (0, 40)
    assert not mo.embedding_grad(torch.zeros(0, 40, device="cuda"), none, 50).any()
    assert mo.embedding_grad(torch.zeros(5, 0, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda"), 50).shape == (50, 0)
    assert mo.embedding(torch.tensor(7, device="cuda"), w).shape == (40,)
