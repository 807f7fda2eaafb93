"""Routing, expert layers and their gradients on the GPU against the float64 oracle.

Tolerances.  u = 2^-24 is half an fp32 step, h half a step of the output's type
(2^-8 for bf16, 2^-24 for fp32), S the sum of the magnitudes of the terms.
  * Products of bf16 operands sum K terms that are exact in fp32: within K 2u S
    of the exact sum whatever the order and however each addition rounds, then
    one rounding h.
  * fp32 operands are three bf16 terms each (exactly); six of the nine products of
    terms are summed, so there are 6 K terms of together at most (1 + 2^-7)^2 S,
    and the three left out are at most 2 2^-24 + 2^-32 of a product, below 3 u: within
    (6 K + 2) 2u 1.02 S.
  * A token's sum of k rows with gates: a product and an addition each, (k + 1) u S.
  * exp in fp32 is taken to be within 4 u; a gate is a quotient of it and a sum of
    n of them: (n + 12) u relative; the difference x - top rounds its argument
    (|x - top| < 64 here): 64 u more.
"""
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


def wide(t):
    return host(t).astype(np.float64)


def rand(g, *size, dtype=BF16, std=1.0):
    return (torch.randn(*size, generator=g) * std).to(dtype).cuda()


def pick(g, tokens, k, experts, drop=0.0):
    """A choice of different experts with an uneven use of them, some slots dropped."""
    score = torch.rand(tokens, experts, generator=g) * torch.rand(experts, generator=g)
    c = torch.argsort(score, dim=1, descending=True)[:, :k].to(torch.int32)
    if c.shape[1] < k:
        c = torch.cat([c, torch.full((tokens, k - c.shape[1]), -1, dtype=torch.int32)], 1)
    c[torch.rand(tokens, k, generator=g) < drop] = -1
    return c.contiguous()


def close(got, want, tol):
    g = wide(got)
    assert g.shape == want.shape
    there = ~np.isnan(want)
    err = np.abs(g - want)[there]
    bad = err > np.broadcast_to(tol, want.shape)[there]
    assert not bad.any() and np.isfinite(g[there]).all(), \
        f"{bad.sum()} of {bad.size} out of tolerance, worst {np.nanmax(err) if err.size else 0}"


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("tokens,k,experts,drop", [
    (0, 2, 4, 0), (1, 1, 1, 0), (1, 6, 64, 0), (5, 3, 2, 0), (64, 6, 64, 0.1), (1000, 1, 7, 0), (1025, 2, 255, 0),
    (700, 3, 256, 0.2), (20000, 2, 512, 0.05), (40000, 1, 3, 0), (333, 64, 100, 0)])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_plan(tokens, k, experts, drop, ids):
    announce(f"plan {tokens} x {k}, {experts} experts, {ids}")
    g = torch.Generator().manual_seed(3)
    choice = pick(g, tokens, k, experts, drop)
    if tokens > 4:
        choice[2, 0], choice[3, 0] = experts, -7            # numbers of no expert
        if k > 1:
            choice[4] = choice[4, 0]                          # one expert many times
    p = mo.expert_plan(choice.to(ids).cuda(), experts)
    c = choice.numpy()
    flat = c.reshape(-1)
    ok = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(ok, flat, experts), kind="stable")
    n = int(ok.sum())
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=experts))])
    place = np.full(flat.size, -1)
    place[order[:n]] = np.arange(n)
    assert np.array_equal(p.offsets.cpu().numpy(), offsets)
    tk = p.tokens.cpu().numpy()
    assert np.array_equal(tk[:n], order[:n] // k) and (tk[n:] == -1).all()
    assert np.array_equal(p.place.cpu().numpy().reshape(-1), place)
    if flat.size <= 500:
        o, t, q = so.plan(c, experts)
        assert np.array_equal(o, offsets) and np.array_equal(t, tk) and np.array_equal(q.reshape(-1), place)


def test_plan_of_many_slots():
    """More than 2^20 slots: four positions a thread."""
    g = torch.Generator().manual_seed(5)
    choice = torch.randint(-1, 100, (300001, 4), generator=g, dtype=torch.int32)
    p = mo.expert_plan(choice.cuda(), 100)
    flat = choice.reshape(-1).numpy()
    order = np.argsort(np.where(flat >= 0, flat, 100), kind="stable")
    n = int((flat >= 0).sum())
    assert int(p.offsets[-1]) == n
    assert np.array_equal(p.tokens.cpu().numpy()[:n], order[:n] // 4)


# ------------------------------------------------------------------ routing
def logits_of(g, tokens, experts, dtype, kind):
    x = torch.randn(tokens, experts, generator=g) * 3
    if kind == "masked" and tokens > 2:
        x[torch.rand(tokens, experts, generator=g) < 0.5] = -np.inf
        x[1] = -np.inf
    if kind == "ties":
        x = torch.round(x / 2)
        x[x == 0] = -0.0
        x[::2][x[::2] == 0] = 0.0
    if kind == "lowest":
        x[torch.rand(tokens, experts, generator=g) < 0.5] = torch.finfo(dtype).min
    return x.to(dtype)


@pytest.mark.parametrize("kind", ["plain", "masked", "ties", "lowest"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 64, 6), (3, 5, 8), (65, 64, 6), (40, 65, 2), (33, 130, 64),
                                              (17, 300, 9), (9, 512, 8)])
def test_route_and_gradient(tokens, experts, k, dtype, kind):
    announce(f"route {tokens} x {experts}, k {k}, {dtype}, {kind}")
    g = torch.Generator().manual_seed(tokens * 7 + experts)
    x = logits_of(g, tokens, experts, dtype, kind)
    xh = x.double().numpy()
    dg = torch.randn(tokens, k, generator=g)
    for normalize in (False, True):
        r = mo.route(x.cuda(), k, normalize=normalize)
        gates, chosen = so.route(xh, k, normalize)
        assert np.array_equal(r.experts.cpu().numpy(), chosen)
        rel = (experts + 12 + 64) * U
        close(r.gates, gates, rel * gates)
        o, t, q = so.plan(chosen, experts)
        assert np.array_equal(r.plan.offsets.cpu().numpy(), o) and np.array_equal(r.plan.tokens.cpu().numpy(), t)
        assert np.array_equal(r.plan.place.cpu().numpy(), q)
        got = mo.route_grad(dg.cuda(), x.cuda(), r)
        assert got.dtype == dtype
        dgh, gh = dg.double().numpy(), wide(r.gates)
        want = so.route_grad(dgh, xh, gh, chosen, normalize)
        # p (dg - sum dg g): the sum has at most k terms, each factor its own error
        live = np.where(chosen >= 0, np.abs(dgh), 0)
        size = (live.max(1) + (live * gh).sum(1))[:, None]
        p = np.zeros(xh.shape)
        for i in range(tokens):
            if normalize:
                for j in range(k):
                    if chosen[i, j] >= 0:
                        p[i, chosen[i, j]] = gh[i, j]
            elif (chosen[i] >= 0).any():
                e = np.exp(xh[i] - xh[i].max())
                p[i] = e / e.sum()
        # the smallest subnormal of either type can be lost in p and in the result
        close(got, want, (2 * rel + (k + 4) * U) * p * size + half(dtype) * np.abs(want) + 2.0 ** -126)


def test_route_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 11, generator=g).double()
    dg = torch.randn(6, 3, generator=g)
    for normalize in (False, True):
        r = mo.route(x.float().cuda(), 3, normalize=normalize)
        got = wide(mo.route_grad(dg.cuda(), x.float().cuda(), r))
        xs, step = x.float().double().numpy(), 1e-5
        for i in range(11):
            up, down = xs.copy(), xs.copy()
            up[:, i] += step
            down[:, i] -= step
            d = ((so.route(up, 3, normalize)[0] - so.route(down, 3, normalize)[0]) * dg.double().numpy()).sum(1) / (2 * step)
            # the difference's own error is of second order: step^2 and rounding / step
            assert np.abs(d - got[:, i]).max() < 1e-5


def test_route_of_rows_that_are_not_finite():
    x = torch.randn(4, 9)
    x[0, 4], x[1, 3], x[2, 7], x[2, 2] = np.nan, np.inf, np.nan, np.inf
    for normalize in (False, True):
        r = mo.route(x.cuda(), 3, normalize=normalize)
        gates, chosen = so.route(x.double().numpy(), 3, normalize)
        assert np.array_equal(r.experts.cpu().numpy(), chosen)
        assert np.isnan(wide(r.gates)[:3]).all() and np.isfinite(wide(r.gates)[3]).all()


def test_route_of_strided_logits():
    x = torch.randn(70, 40)
    a = mo.route(x.cuda()[:, 3:24], 2)
    b = mo.route(x[:, 3:24].contiguous().cuda(), 2)
    assert torch.equal(a.gates, b.gates) and torch.equal(a.experts, b.experts) and torch.equal(a.plan.tokens, b.plan.tokens)


# ------------------------------------------------------------------ products
def check_layer(tokens, k, experts, cols, outs, dtype, gather, drop=0.0, seed=1, out_dtype=None):
    announce(f"experts {tokens} x {k} of {experts}, {cols} -> {outs}, {dtype}, gather {gather}")
    g = torch.Generator().manual_seed(seed)
    choice = pick(g, tokens, k, experts, drop)
    plan = mo.expert_plan(choice.cuda(), experts)
    n = tokens * k
    x, w = rand(g, tokens if gather else n, cols, dtype=dtype), rand(g, experts, outs, cols, dtype=dtype)
    dy = rand(g, n, outs, dtype=dtype)
    offsets, tk, _ = so.plan(choice.numpy(), experts)
    xs = so.rows_of(wide(x), tk) if gather else wide(x)
    ws, dys = wide(w).reshape(experts, outs, cols), wide(dy)
    y = mo.expert_linear(x, w, plan, gather=gather, dtype=out_dtype)
    dx, dw = mo.expert_linear_grad(dy, w, x, plan, gather=gather)
    ot = out_dtype or dtype
    assert y.dtype == ot and dx.dtype == dtype and dw.dtype == F32 and dw.shape == (experts, outs, cols)

    def tol(depth, s, want, t):
        c = depth * 2 * U if dtype == BF16 else (6 * depth + 2) * 2 * U * 1.02
        return c * s + half(t) * (np.abs(want) + c * s)
    want, s = so.linear(xs, ws, offsets), so.linear(np.abs(xs), np.abs(ws), offsets)
    close(y, want, tol(cols, s, want, ot))
    (wdx, wdw), (sdx, sdw) = so.linear_grad(dys, ws, xs, offsets), so.linear_grad(np.abs(dys), np.abs(ws), np.abs(xs), offsets)
    close(dx, wdx, tol(outs, sdx, wdx, dtype))
    depth = np.diff(offsets)[:, None, None]
    close(dw, wdw, tol(depth, sdw, wdw, F32))
    return x, w, dy, plan, y, dx, dw


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,k,experts,cols,outs", [
    (1, 1, 1, 1, 1), (1, 2, 8, 8, 16), (7, 2, 3, 24, 40), (8, 6, 64, 136, 96), (40, 1, 5, 65, 33), (130, 2, 4, 33, 7),
    (300, 2, 3, 200, 264), (300, 1, 1, 128, 520), (517, 3, 9, 77, 129), (270, 2, 70, 64, 72)])
def test_products(tokens, k, experts, cols, outs, dtype, gather):
    check_layer(tokens, k, experts, cols, outs, dtype, gather)


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("tokens,k,experts,cols,outs,dtype", [
    (300, 2, 3, 200, 264, BF16), (520, 1, 1, 128, 520, BF16), (90, 3, 9, 77, 129, BF16), (300, 2, 3, 200, 264, F32),
    (33, 2, 70, 48, 40, BF16), (1300, 1, 2, 712, 288, BF16)])
def test_products_by_every_tile(tokens, k, experts, cols, outs, dtype, tile, monkeypatch):
    monkeypatch.setenv("MUON_EXPERT_TILE", str(tile))
    for gather in (False, True):
        check_layer(tokens, k, experts, cols, outs, dtype, gather, drop=0.1)


@pytest.mark.parametrize("tile", [64, 128, 256])
def test_many_tiles_a_block(tile, monkeypatch):
    """More tiles than blocks, so that a block goes from tile to tile: against the sums of fp32 products
    in float64, on the GPU."""
    monkeypatch.setenv("MUON_EXPERT_TILE", str(tile))
    g = torch.Generator().manual_seed(tile)
    experts, cols, outs, tokens = (5, 320, 1160, 13000) if tile == 256 else (5, 136, 456, 6000)
    choice = pick(g, tokens, 2, experts)
    plan = mo.expert_plan(choice.cuda(), experts)
    x, w, dy = rand(g, tokens, cols), rand(g, experts, outs, cols), rand(g, 2 * tokens, outs)
    y = mo.expert_linear(x, w, plan, gather=True)
    dx, dw = mo.expert_linear_grad(dy, w, x, plan, gather=True)
    at = plan.offsets.tolist()
    xs = x[plan.tokens.long()].double()
    for e in range(experts):
        r = slice(at[e], at[e + 1])
        for got, a, b in ((y[r], xs[r], w[e].double().t().contiguous()), (dx[r], dy[r].double(), w[e].double()),
                          (dw[e], dy[r].double().t().contiguous(), xs[r])):
            want, s = torch.mm(a, b), torch.mm(a.abs(), b.abs())
            tol = a.shape[1] * 2 * U * s
            tol = tol + half(got.dtype) * (want.abs() + tol)
            assert ((got.double() - want).abs() <= tol).all(), (tile, e)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_with_dropped_slots(dtype):
    check_layer(200, 3, 6, 72, 104, dtype, True, drop=0.3)
    check_layer(50, 2, 4, 16, 24, dtype, False, drop=1.0)   # no slot is left


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_of_other_output_types(dtype):
    check_layer(60, 2, 3, 40, 56, dtype, True, out_dtype=F32 if dtype == BF16 else BF16)


def test_no_tokens_and_empty_features():
    plan = mo.expert_plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    w = torch.randn(3, 16, 8, device="cuda", dtype=BF16)
    x, dy = torch.zeros(0, 8, device="cuda", dtype=BF16), torch.zeros(0, 16, device="cuda", dtype=BF16)
    assert mo.expert_linear(x, w, plan).shape == (0, 16)
    dx, dw = mo.expert_linear_grad(dy, w, x, plan)
    assert dx.shape == (0, 8) and not dw.any() and dw.shape == (3, 16, 8)
    plan = mo.expert_plan(torch.tensor([[0], [2]], device="cuda"), 3)
    y = mo.expert_linear(torch.zeros(2, 0, device="cuda", dtype=BF16), w[:, :, :0], plan)
    assert y.shape == (2, 16) and not y.any()


def test_fp32_products_keep_24_bits():
    """Of one and two terms, where leaving out any of the six products shows."""
    for cols in (1, 2):
        check_layer(400, 1, 2, cols, 130, F32, False, seed=9)


@pytest.mark.parametrize("dtype,cols,outs", [(BF16, 64, 72), (BF16, 33, 41), (F32, 40, 24)])
def test_strided_operands_and_outputs(dtype, cols, outs):
    """Column slices, matrices and rows apart, outputs that neighbours share a buffer with."""
    g = torch.Generator().manual_seed(2)
    plan = mo.expert_plan(pick(g, 90, 2, 4).cuda(), 4)
    for off in (8, 3):
        xb, wb, yb = rand(g, 90, cols + 16, dtype=dtype), rand(g, 5, outs + 3, cols + 24, dtype=dtype), rand(g, 180, outs + 16, dtype=dtype)
        x, w, dy = xb[:, off:off + cols], wb[:4, 1:outs + 1, off:off + cols], yb[:, off:off + outs]
        xc, wc, dyc = x.contiguous(), w.contiguous(), dy.contiguous()
        ref = mo.expert_linear(xc, wc, plan, gather=True)
        room = torch.full((180, outs + 16), 7.0, dtype=dtype, device="cuda")
        got = mo.expert_linear(x, w, plan, gather=True, out=room[:, off:off + outs])
        assert torch.equal(got, ref) and (room[:, :off] == 7).all() and (room[:, off + outs:] == 7).all()
        dx, dw = mo.expert_linear_grad(dyc, wc, xc, plan, gather=True)
        room = torch.full((4, outs + 3, cols + 24), 7.0, device="cuda")
        dx2, dw2 = mo.expert_linear_grad(dy, w, x, plan, gather=True, out=room[:, 2:outs + 2, off:off + cols])
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        assert (room[:, :2] == 7).all() and (room[:, outs + 2:] == 7).all() and (room[:, :, :off] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_the_last_expert_are_left_alone(dtype):
    g = torch.Generator().manual_seed(4)
    choice = pick(g, 300, 2, 3, drop=0.5)
    plan = mo.expert_plan(choice.cuda(), 3)
    n = int(plan.offsets[-1])
    assert 0 < n < 600
    x, w = rand(g, 600, 64, dtype=dtype), rand(g, 3, 48, 64, dtype=dtype)
    x[n:] = np.nan                                            # nor are they read
    out = torch.full((600, 48), 5.0, dtype=dtype, device="cuda")
    mo.expert_linear(x, w, plan, out=out)
    assert (out[n:] == 5).all() and torch.isfinite(out[:n]).all()
    dy = rand(g, 600, 48, dtype=dtype)
    dy[n:] = np.nan
    dx, dw = mo.expert_linear_grad(dy, w, x, plan)
    assert torch.isfinite(dw).all() and torch.isfinite(dx[:n]).all()
    t = rand(g, 300, 40, dtype=dtype)
    rows = torch.full((600, 40), 5.0, dtype=dtype, device="cuda")
    mo.expert_gather(t, plan, out=rows)
    assert torch.equal(rows[:n], t[plan.tokens[:n].long()]) and (rows[n:] == 5).all()


@pytest.mark.parametrize("cols,outs", [(64, 64), (70, 61)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_finite_stays_with_its_expert(dtype, cols, outs):
    """NaN in one expert's rows and matrices reaches no other expert's results."""
    g = torch.Generator().manual_seed(6)
    choice = torch.arange(90, dtype=torch.int32).reshape(-1, 1) % 3
    plan = mo.expert_plan(choice.cuda(), 3)
    x, w, dy = rand(g, 90, cols, dtype=dtype), rand(g, 3, outs, cols, dtype=dtype), rand(g, 90, outs, dtype=dtype)
    x[30:60], w[1], dy[30:60] = np.nan, np.nan, np.inf
    y = mo.expert_linear(x, w, plan)
    dx, dw = mo.expert_linear_grad(dy, w, x, plan)
    for t in (y, dx):
        assert torch.isfinite(t[:30]).all() and torch.isfinite(t[60:]).all() and torch.isnan(t[30:60]).all()
    assert torch.isfinite(dw[[0, 2]]).all() and torch.isnan(dw[1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("grad", [BF16, F32])
def test_accumulated_gradients(dtype, grad):
    g = torch.Generator().manual_seed(8)
    plan = mo.expert_plan(pick(g, 70, 2, 5).cuda() % 4, 5)    # the last expert has no rows
    x, dy = rand(g, 70, 64, dtype=dtype), rand(g, 140, 40, dtype=dtype)
    _, dw = mo.expert_linear_grad(dy, None, x, plan, gather=True)
    old = rand(g, 5, 40, 64, dtype=grad)
    out = old.clone()
    _, got = mo.expert_linear_grad(dy, None, x, plan, gather=True, out=out, accumulate=True)
    assert got is out and torch.equal(out, (old.float() + dw).to(grad))
    assert torch.equal(out[4], old[4])
    _, plain = mo.expert_linear_grad(dy, None, x, plan, gather=True, out=out)
    assert torch.equal(plain, dw.to(grad))


SPLIT = [(2100, 1, 2, 100, 60), (1600, 2, 2, 64, 64), (3001, 1, 1, 33, 77), (8000, 2, 4, 64, 136)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,k,experts,cols,outs", SPLIT)
def test_split_contractions(tokens, k, experts, cols, outs, dtype, gather):
    """Few tiles and many rows: parts of an expert's rows are summed apart, then in order."""
    x, _, dy, plan, _, _, dw = check_layer(tokens, k, experts, cols, outs, dtype, gather, drop=0.1)
    desc = mo.experts._stack(dw, dw.device)
    assert mo._lib.load().muon_expert_linear_dw_workspace_bytes(tokens * k, desc) > 0
    for _ in range(3):
        assert torch.equal(mo.expert_linear_grad(dy, None, x, plan, gather=gather)[1], dw)


@pytest.mark.parametrize("grad", [BF16, F32])
@pytest.mark.parametrize("off,cols,outs", [(0, 64, 40), (3, 61, 40)])
def test_split_contractions_accumulated(off, cols, outs, grad):
    """Into strided matrices, with all rows at one expert, NaN behind the last and in a part of the memory used."""
    g = torch.Generator().manual_seed(9)
    choice = torch.full((4000, 1), 1, dtype=torch.int32)
    choice[::7] = -1
    choice[:5] = 2
    plan = mo.expert_plan(choice.cuda(), 4)
    x, dy = rand(g, 4000, cols), rand(g, 4000, outs)
    n = int(plan.offsets[-1])
    x[n:], dy[n:] = np.nan, np.nan
    _, dw = mo.expert_linear_grad(dy, None, x, plan)
    assert mo._lib.load().muon_expert_linear_dw_workspace_bytes(4000, mo.experts._stack(dw, dw.device)) > 0
    assert (dw[[0, 3]] == 0).all() and torch.isfinite(dw).all() and (dw[1:3] != 0).any()
    room = rand(g, 4, outs + 1, cols + off + 5, dtype=grad)
    old = room.clone()
    out = room[:, 1:, off:off + cols]
    mo.expert_linear_grad(dy, None, x, plan, out=out, accumulate=True)
    want = old.clone()
    want[:, 1:, off:off + cols] = (old[:, 1:, off:off + cols].float() + dw).to(grad)
    assert torch.equal(room, want)
    mo.expert_linear_grad(dy, None, x, plan, out=out)
    want[:, 1:, off:off + cols] = dw.to(grad)
    assert torch.equal(room, want)
    x[n - 1] = np.nan                                         # of expert 2
    _, dw = mo.expert_linear_grad(dy, None, x, plan)
    assert torch.isfinite(dw[[0, 1, 3]]).all() and torch.isnan(dw[2]).all()


def test_split_contractions_in_a_graph():
    """Captured, replayed with other rows and another choice, beside eager calls on another stream."""
    g = torch.Generator().manual_seed(10)
    choice = pick(g, 4000, 1, 3, drop=0.1).cuda()
    x, dy = rand(g, 4000, 72), rand(g, 4000, 56)

    def grads():
        plan = mo.expert_plan(choice, 3)
        return mo.expert_linear_grad(dy, None, x, plan, gather=True)[1]
    assert mo._lib.load().muon_expert_linear_dw_workspace_bytes(4000, mo.experts._stack(grads(), x.device)) > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dw = grads()
    for i in range(4):
        choice.copy_(pick(g, 4000, 1, 3, drop=0.2 * i))
        x.copy_(rand(g, 4000, 72))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            want = grads()
        torch.cuda.synchronize()
        assert torch.equal(dw, want) and (dw != 0).any(), i


def test_gradients_against_differences():
    """d/dw and d/dx of sum(dy y) in fp32, whose error over a difference of 0.5 is that of the sums."""
    g = torch.Generator().manual_seed(10)
    plan = mo.expert_plan(pick(g, 12, 2, 3).cuda(), 3)
    x, w, dy = rand(g, 24, 6, dtype=F32), rand(g, 3, 5, 6, dtype=F32), rand(g, 24, 5, dtype=F32)
    dx, dw = mo.expert_linear_grad(dy, w, x, plan)

    def value(xx, ww):
        return float((mo.expert_linear(xx, ww, plan).double() * dy.double()).sum())
    # linear in each: the difference is exact but for roundings, 24 rows x 5 x 6 terms
    tol = 24 * 5 * (6 * 6 + 2) * 2 * U * float(x.abs().max() * w.abs().max() * dy.abs().max())
    for e, i, j in [(0, 0, 0), (1, 4, 5), (2, 2, 3)]:
        up, down = w.clone(), w.clone()
        up[e, i, j] += 0.5
        down[e, i, j] -= 0.5
        assert abs(value(x, up) - value(x, down) - float(dw[e, i, j])) < 4 * tol
    for r, j in [(0, 0), (11, 3), (23, 5)]:
        up, down = x.clone(), x.clone()
        up[r, j] += 0.5
        down[r, j] -= 0.5
        assert abs(value(up, w) - value(down, w) - float(dx[r, j])) < 4 * tol


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,k,experts,cols,drop", [(1, 1, 1, 1, 0), (8, 6, 64, 200, 0), (130, 3, 5, 77, 0.3),
                                                        (50, 20, 30, 520, 0.1), (3, 2, 4, 1033, 1.0)])
def test_combine_and_gradient(tokens, k, experts, cols, drop, dtype):
    announce(f"combine {tokens} x {k}, {cols}, {dtype}")
    g = torch.Generator().manual_seed(tokens)
    choice = pick(g, tokens, k, experts, drop)
    plan = mo.expert_plan(choice.cuda(), experts)
    place = so.plan(choice.numpy(), experts)[2]
    y, dout = rand(g, tokens * k, cols, dtype=dtype), rand(g, tokens, cols, dtype=dtype)
    gates = torch.rand(tokens, k, generator=g).cuda()
    yh, dh, gh = wide(y), wide(dout), wide(gates)
    for gt, gw in ((gates, gh), (None, np.ones_like(gh))):
        want, s = so.combine(yh, gw, place), so.combine(np.abs(yh), np.abs(gw), place)
        close(mo.expert_combine(y, plan, gt), want, (k + 1) * U * s * (1 + half(dtype)) + half(dtype) * np.abs(want))
    dy, dg = mo.expert_combine_grad(dout, y, plan, gates)
    wdy, wdg = so.combine_grad(dh, yh, gh, place)
    close(dy, wdy, (U + half(dtype)) * np.abs(wdy) * (1 + U))
    close(dg, wdg, (cols + 1) * 2 * U * so.combine_grad(np.abs(dh), np.abs(yh), gh, place)[1])


def test_combine_of_strided_rows():
    g = torch.Generator().manual_seed(12)
    plan = mo.expert_plan(pick(g, 40, 2, 4).cuda(), 4)
    y, dout, gates = rand(g, 80, 50), rand(g, 40, 60), torch.rand(40, 2, generator=g).cuda()
    ref = mo.expert_combine(y[:, 3:36].contiguous(), plan, gates)
    room = torch.full((40, 50), 3.0, dtype=BF16, device="cuda")
    got = mo.expert_combine(y[:, 3:36], plan, gates, out=room[:, 5:38])
    assert torch.equal(got, ref) and (room[:, :5] == 3).all() and (room[:, 38:] == 3).all()
    a = mo.expert_combine_grad(dout[:, 1:34], y[:, 3:36], plan, gates)
    b = mo.expert_combine_grad(dout[:, 1:34].contiguous(), y[:, 3:36].contiguous(), plan, gates)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
