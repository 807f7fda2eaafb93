"""Expert layers and the embedding on the GPU where indexes, ranges and strides are unusual."""
import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import experts as ex
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


def wide(t):
    return host(t).astype(np.float64)


def mat(t):
    return ex._MAT1.pack(*ex._mat(t, t.device))


def overwritten_plan(g):
    """50 tokens x 2: slots with places of no row, of another token's row, two at one row, and rows of no token."""
    plan = mo.expert_plan(torch.randint(0, 4, (50, 2), generator=g).cuda(), 4)
    place, tokens = plan.place.cpu(), plan.tokens.cpu()
    place[1] = torch.tensor([100, -5])
    place[2] = torch.tensor([(1 << 31) - 1, -(1 << 31)])
    place[3, 0] = place[4, 0]
    place[5, 1] = place[5, 0]
    tokens[place[6, 0]] = 50
    tokens[place[7, 1]] = -(1 << 31)
    plan.place.copy_(place)
    plan.tokens.copy_(tokens)
    return plan, place.numpy(), tokens.numpy()


@pytest.mark.parametrize("cols", [16, 24, 33])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_of_a_sum_over_a_plan_that_was_written_over(dtype, cols):
    """Every gate has a gradient, 0 where its slot has no row of its token's; rows of no slot are left alone."""
    announce(f"combine_grad of an overwritten plan, {dtype}, {cols}")
    g = torch.Generator().manual_seed(cols)
    plan, place, tokens = overwritten_plan(g)
    y, dout = (torch.randn(n, cols, generator=g).to(dtype).cuda() for n in (100, 50))
    gates = torch.rand(50, 2, generator=g).cuda()
    yh, dh, gh = wide(y), wide(dout), wide(gates)
    want, size, rows = np.zeros((50, 2)), np.zeros((50, 2)), np.zeros((100, 1))
    for t in range(50):
        for j in range(2):
            p = place[t, j]
            if 0 <= p < 100 and tokens[p] == t:
                want[t, j], size[t, j] = dh[t] @ yh[p], np.abs(dh[t]) @ np.abs(yh[p])
                rows[p] += gh[t, j]
    dy, dg = torch.full((100, cols), 7.0, dtype=dtype, device="cuda"), torch.full((50, 2), torch.nan, device="cuda")
    ex._call("muon_expert_combine_grad", dy.device, mat(dout), mat(y), gates.data_ptr(), plan.desc, mat(dy), dg.data_ptr())
    assert (np.abs(wide(dg) - want) <= (cols + 1) * 2 * U * size).all()
    wdy = rows * dh[np.clip(tokens, 0, 49)]
    mine = rows[:, 0] > 0
    # the gates of two slots at one row are added first: a rounding more
    assert (np.abs(wide(dy) - wdy) <= (2 * U + half(dtype)) * np.abs(wdy) * (1 + 2 * U))[mine].all()
    assert 0 < (~mine).sum() < 10 and (dy[torch.from_numpy(~mine).cuda()] == 7).all()
    # the same numbers where they are all that is asked for
    only = torch.full((50, 2), torch.nan, device="cuda")
    ex._call("muon_expert_combine_grad", dy.device, mat(dout), mat(y), gates.data_ptr(), plan.desc, None, only.data_ptr())
    assert torch.equal(only, dg)


@pytest.mark.parametrize("cols", [16, 33])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_gathered_by_a_plan_that_was_written_over(dtype, cols):
    """Each row is its token's, whatever the places hold, as in a product that gathers; no token's are left alone."""
    announce(f"gather by an overwritten plan, {dtype}, {cols}")
    g = torch.Generator().manual_seed(cols)
    plan, place, tokens = overwritten_plan(g)
    x = torch.randn(50, cols, generator=g).to(dtype).cuda()
    room = torch.full((102, cols), 7.0, dtype=dtype, device="cuda")
    mo.expert_gather(x, plan, out=room[1:101])
    ok = (tokens >= 0) & (tokens < 50)
    assert ok.sum() == 98
    want = torch.full((102, cols), 7.0, dtype=dtype, device="cuda")
    want[1:101][torch.from_numpy(ok).cuda()] = x[torch.from_numpy(tokens[ok]).long().cuda()]
    assert torch.equal(room, want)


def test_ids_and_choices_of_any_row_pitch():
    """A language model's inputs and targets, as slices of one batch; also captured."""
    g = torch.Generator().manual_seed(7)
    batch, w = torch.randint(0, 60, (9, 65), generator=g).cuda(), torch.randn(60, 40, generator=g).cuda()
    for ids in (batch[:, :-1], batch[:, 1:], batch.int()[:, 3:], batch[::2], batch[0].expand(3, 65)):
        dense = ids.contiguous()
        dy = torch.randn(*ids.shape, 40, generator=g).cuda()
        assert torch.equal(mo.embedding(ids, w), w[dense])
        assert torch.equal(mo.embedding_grad(dy, ids, 60), mo.embedding_grad(dy, dense, 60))
    choice = torch.randint(-1, 5, (700, 6), generator=g).cuda()
    a, b = mo.expert_plan(choice[:, 1:4], 5), mo.expert_plan(choice[:, 1:4].contiguous(), 5)
    assert torch.equal(a.buffer, b.buffer)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = mo.embedding(batch[:, :-1], w)
    for _ in range(3):
        batch.copy_(torch.randint(0, 60, (9, 65), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mo.embedding(batch[:, :-1].contiguous(), w))
