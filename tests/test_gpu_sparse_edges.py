"""Expert layers and the embedding on the GPU where indexes, ranges and strides are unusual."""
import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from oracle import sparse_oracle as so
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


def products_in_float64(x, w, dy, offsets):
    return so.linear(x, w, offsets), *so.linear_grad(dy, w, x, offsets)


@pytest.mark.parametrize("power", [0, 60, 100, 105, 110, 112, 116, 118, 120, 124, 126, 130, 137, 149])
@pytest.mark.parametrize("cols,outs,rows", [(1, 3, 5), (2, 40, 9), (77, 129, 150), (64, 64, 700)])
def test_fp32_products_of_small_numbers(cols, outs, rows, power):
    """Operands of 2^-power times operands of order 1, subnormal ones among them, in each place.

    The bound of the products of fp32, (6 K + 2) 2u 1.02 S, and for sums among the subnormal numbers, of which
    one step is 2^-149: a step for each of K first terms' products, 2^-8 of one for each of 2 K and 2^-16 for each
    of 3 K others, and one each for the sums' addition and its two products: (2 K + 4) 2^-149 in all."""
    announce(f"fp32 products of 2^-{power}: {rows} rows, {cols} -> {outs}")
    g = torch.Generator().manual_seed(power + cols)
    plan = mo.expert_plan((torch.arange(rows, dtype=torch.int32) % 3).reshape(-1, 1).cuda(), 3)
    offsets = plan.offsets.cpu().numpy()

    def rand(*size, small=False):
        t = torch.randn(*size, generator=g).double() * (2.0 ** -power if small else 1.0)
        return t.float().cuda()
    for which in range(3):
        x, w, dy = (rand(*s, small=i == which) for i, s in enumerate(((rows, cols), (3, outs, cols), (rows, outs))))
        got = (mo.expert_linear(x, w, plan), *mo.expert_linear_grad(dy, w, x, plan))
        xh, wh, dh = wide(x), wide(w).reshape(3, outs, cols), wide(dy)
        want = products_in_float64(xh, wh, dh, offsets)
        size = products_in_float64(np.abs(xh), np.abs(wh), np.abs(dh), offsets)
        depth = (cols, outs, np.diff(offsets)[:, None, None])
        for a, b, s, k in zip(got, want, size, depth):
            tol = (6 * k + 2) * 2 * U * 1.02 * s + U * np.abs(b) + (2 * k + 4) * 2.0 ** -149
            assert (np.abs(wide(a) - b) <= tol).all(), (which, np.max(np.abs(wide(a) - b) / tol))


@pytest.mark.parametrize("cols,outs", [(8, 40), (77, 129)])
def test_fp32_products_of_infinities_and_large_numbers(cols, outs):
    """An infinity's products are infinities, NaN with zeros and with each other's opposites; no other result changes."""
    g = torch.Generator().manual_seed(cols)
    plan = mo.expert_plan(torch.zeros(90, 1, dtype=torch.int32).cuda(), 1)
    x, w = torch.randn(90, cols, generator=g), torch.randn(1, outs, cols, generator=g)
    x[3, 2], x[5, 0], x[7, 1], x[7, 3], x[9, 4] = np.inf, -np.inf, np.inf, -np.inf, np.nan
    w[0, 6, 2] = 0.0
    x[11], x[12, 5] = 1e38, 3.4e38                            # sums that overflow, and a number that counts as infinite
    w[0, 8, 1] = np.inf
    got = mo.expert_linear(x.cuda(), w.cuda(), plan).cpu()
    x[12, 5] = np.inf
    want = x.double() @ w[0].double().t()
    plain = [r for r in range(90) if r not in (3, 5, 7, 9, 11, 12)]
    for r in (3, 5, 7, 9, 12):
        assert torch.equal(got[r].isnan(), want[r].isnan()) and torch.equal(got[r].isinf(), want[r].isinf()), r
        ok = ~want[r].isnan()
        assert torch.equal(got[r][ok].double(), want[r][ok]), r
    assert got[3, 6].isnan() and got[7].isnan().sum() >= outs // 4
    assert not got[11][want[11].abs() > 1e39].isfinite().any()
    s = x.double().abs() @ w[0].double().abs().t()
    cols_ok = [c for c in range(outs) if c != 8]
    err = (got.double() - want).abs()[plain][:, cols_ok]
    assert (err <= ((6 * cols + 2) * 2.04 * U * s + U * want.abs())[plain][:, cols_ok]).all()
    assert torch.equal(got[plain][:, 8].double(), want[plain][:, 8])
    big = (torch.rand(90, cols, generator=g) + 1) * 1e38     # 1e38 .. 2e38, sums below 2^127
    small = torch.randn(1, outs, cols, generator=g) / (8 * cols)
    got = mo.expert_linear(big.cuda(), small.cuda(), plan).cpu()
    want, s = big.double() @ small[0].double().t(), big.double() @ small[0].double().abs().t()
    assert ((got.double() - want).abs() <= (6 * cols + 2) * 2.04 * U * s + U * want.abs()).all()


@pytest.mark.parametrize("dtype,off", [(BF16, 8), (BF16, 3), (F32, 4), (F32, 1)])
def test_tokens_rows_that_span_gigabytes(dtype, off):
    """Gathered rows between 2 GiB and what a product addresses, and past it, where they are sorted first:
    the same bits as from rows that lie together."""
    pitch = (1 << 21) // dtype.itemsize                       # 2 MiB from row to row
    most = mo._lib.GATHER_BYTES >> 21                         # rows of as much
    g = torch.Generator().manual_seed(off)
    room = torch.empty((most + 40) * pitch, dtype=dtype, device="cuda")
    for rows in (most, most + 1, most + 40):
        announce(f"{rows} rows 2 MiB apart, {dtype}, offset {off}")
        x = room.as_strided((rows, 72), (pitch, 1), off)
        near = torch.randn(rows, 72, generator=g).to(dtype).cuda()
        x.copy_(near)
        choice = torch.full((rows, 2), -1, dtype=torch.int32)
        choice[rows // 2 + 100:] = torch.randint(0, 3, (rows - rows // 2 - 100, 2), generator=g, dtype=torch.int32)
        plan = mo.expert_plan(choice.cuda(), 3)
        n = int(plan.offsets[-1])
        assert n > 1500 and int(plan.tokens[:n].min()) * pitch * dtype.itemsize > 1 << 31
        w, dy = torch.randn(3, 56, 72, generator=g).to(dtype).cuda(), torch.randn(2 * rows, 56, generator=g).to(dtype).cuda()
        assert torch.equal(mo.expert_linear(x, w, plan, gather=True)[:n], mo.expert_linear(near, w, plan, gather=True)[:n])
        a, b = (mo.expert_linear_grad(dy, None, t, plan, gather=True)[1] for t in (x, near))
        assert torch.equal(a, b) and (a != 0).all()
        assert torch.equal(mo.expert_gather(x, plan)[:n], near[plan.tokens[:n].long()])
        ids = torch.randint(rows // 2, rows, (300,), generator=g).cuda()
        assert torch.equal(mo.embedding(ids, x), near[ids])


@pytest.mark.parametrize("experts,slots", [(64, 1 << 18), (64, (1 << 18) + 1), (512, 1 << 17), (512, (1 << 17) + 1),
                                           (512, (1 << 18) + 4097)])
def test_plans_around_the_sorts_borders(experts, slots):
    """One position a thread and four, in keys of 8 and of 10 bits."""
    announce(f"plan {slots} of {experts}")
    g = torch.Generator().manual_seed(slots)
    choice = torch.randint(-1, experts + 1, (slots, 1), generator=g, dtype=torch.int32)
    plan = mo.expert_plan(choice.cuda(), experts)
    flat = choice.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order, n = torch.argsort(key, stable=True), int((key < experts).sum())
    assert torch.equal(plan.offsets.cpu().long(), torch.cumsum(torch.bincount(key + 1, minlength=experts + 2), 0)[:experts + 1])
    assert torch.equal(plan.tokens.cpu()[:n].long(), order[:n]) and (plan.tokens[n:] == -1).all()
    place = torch.full((slots,), -1, dtype=torch.int64)
    place[order[:n]] = torch.arange(n)
    assert torch.equal(plan.place.cpu().reshape(-1).long(), place)
