"""Embedding, routing, expert layers and their gradients as a program uses them: one
after the other into the optimizers' steps, captured and replayed, on other streams,
from several threads, over and over.

The layers run on small whole numbers, so that every product and sum is exact in fp32
and bf16 and results are compared bit for bit with integer arithmetic."""
import threading

import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def whole(g, *size, most=1):
    return torch.randint(-most, most + 1, size, generator=g)


def layer(ids, table, choice, gates, w1, w2, dout, experts):
    """A table's rows through two layers of experts with a relu between and back:
    output, gradients of the table, both layers and the gates."""
    plan = mo.expert_plan(choice, experts)
    x = mo.embedding(ids, table)
    h = mo.expert_linear(x, w1, plan, gather=True)
    a = torch.relu(h)
    y = mo.expert_linear(a, w2, plan)
    out = mo.expert_combine(y, plan, gates)
    dy, dgates = mo.expert_combine_grad(dout, y, plan, gates)
    da, dw2 = mo.expert_linear_grad(dy, w2, a, plan)
    dh = torch.where(h > 0, da, torch.zeros_like(da))
    dx, dw1 = mo.expert_linear_grad(dh, w1, x, plan, gather=True)
    dtable = mo.embedding_grad(mo.expert_combine(dx, plan), ids, table.shape[0])
    return out, dtable, dw1, dw2, dgates


def layer_in_integers(ids, table, choice, gates, w1, w2, dout):
    """The same token by token, in int64 on the host."""
    dtable, dw1, dw2 = torch.zeros_like(table), torch.zeros_like(w1), torch.zeros_like(w2)
    out, dgates = torch.zeros_like(dout), torch.zeros_like(gates)
    for t, i in enumerate(ids.tolist()):
        x = table[i] if i >= 0 else torch.zeros_like(table[0])
        dx = torch.zeros_like(x)
        for j, e in enumerate(choice[t].tolist()):
            if e < 0:
                continue
            h = w1[e] @ x
            a = h.clamp(min=0)
            y = w2[e] @ a
            out[t] += gates[t, j] * y
            dgates[t, j] = dout[t] @ y
            dy = gates[t, j] * dout[t]
            dw2[e] += torch.outer(dy, a)
            dh = (w2[e].t() @ dy) * (h > 0)
            dw1[e] += torch.outer(dh, x)
            dx += w1[e].t() @ dh
        if i >= 0:
            dtable[i] += dx
    return out, dtable, dw1, dw2, dgates


def problem(seed, tokens=70, k=2, experts=5, vocab=40, cols=24, wide=40):
    g = torch.Generator().manual_seed(seed)
    choice = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)])
    choice[3] = -1                                            # a token of padding
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    ids[3] = -1
    # one in eight weights is not 0, so that sums stay below 2^8 (whole numbers in bf16)
    sparse = lambda *s: whole(g, *s) * (torch.rand(*s, generator=g) < 0.125)
    return (ids, whole(g, vocab, cols), choice, torch.randint(1, 3, (tokens, k), generator=g), sparse(experts, wide, cols),
            sparse(experts, cols, wide), whole(g, tokens, cols) * (torch.rand(tokens, cols, generator=g) < 0.25))


def on_gpu(p, dtype):
    ids, table, choice, gates, w1, w2, dout = p
    return (ids.cuda(), table.to(dtype).cuda(), choice.to(torch.int32).cuda(), gates.float().cuda(), w1.to(dtype).cuda(),
            w2.to(dtype).cuda(), dout.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [dict(), dict(tokens=300, k=3, experts=4, cols=33, wide=21), dict(tokens=1, k=1, experts=1)])
def test_a_layer_and_its_gradients_in_whole_numbers(dtype, shape):
    p = problem(1, **shape) if shape.get("tokens") != 1 else None
    if p is None:
        g = torch.Generator().manual_seed(2)
        p = (torch.tensor([3]), whole(g, 8, 16), torch.tensor([[0]]), torch.tensor([[2]]), whole(g, 1, 24, 16), whole(g, 1, 16, 24), whole(g, 1, 16))
    want = layer_in_integers(*p)
    assert all(w.abs().max() < 2 ** 24 for w in want)
    if dtype == BF16:   # what is stored in bf16 between the calls has to be whole there: at most 8 bits
        q = layer_in_integers(*p[:6], p[6])
        assert q[0].abs().max() <= 256
    got = layer(*on_gpu(p, dtype), p[4].shape[0])
    for name, a, b in zip(("out", "dtable", "dw1", "dw2", "dgates"), got, want):
        assert torch.equal(a.double().cpu(), b.double()), name


def test_gradients_go_to_the_optimizers():
    """list(dw) are gradients for Muon.step, the table's and the router's for AdamW.step."""
    p = problem(5, cols=32, wide=48)
    ids, table, choice, gates, w1, w2, dout = on_gpu(p, BF16)
    out, dtable, dw1, dw2, _ = layer(ids, table, choice, gates, w1, w2, dout, 5)
    ref = layer_in_integers(*p)
    results = []
    for grads, dt in (((list(dw1) + list(dw2)), dtable),
                      ([t.float().cuda() for t in list(ref[2]) + list(ref[3])], ref[1].float().cuda())):
        a, b, tab = w1.clone(), w2.clone(), table.clone()
        mats = list(a) + list(b)                              # views: the step writes the stacks
        muon, adamw = mo.Muon(mats, lr=0.02), mo.AdamW([tab], lr=1e-3)
        for _ in range(2):
            muon.step(grads)
            adamw.step([dt])
        assert not torch.equal(a, w1) and not torch.equal(tab, table)
        results.append((a, b, tab))
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_a_router_in_the_run():
    """route's gates and plan through the layer: the same as its choice given by hand."""
    g = torch.Generator().manual_seed(9)
    x, wr = torch.randn(200, 48, generator=g).cuda(), torch.randn(6, 48, generator=g).cuda()
    w = torch.randn(6, 40, 48, generator=g).cuda()
    logits = x @ wr.t()
    r = mo.route(logits, 2, normalize=True)
    plan = mo.expert_plan(r.experts, 6)
    for a, b in ((r.plan.offsets, plan.offsets), (r.plan.tokens, plan.tokens), (r.plan.place, plan.place)):
        assert torch.equal(a, b)
    y = mo.expert_linear(x, w, r.plan, gather=True)
    out = mo.expert_combine(y, r.plan, r.gates)
    assert torch.equal(y, mo.expert_linear(mo.expert_gather(x, plan), w, plan))
    dout = torch.randn(200, 40, generator=g).cuda()
    _, dgates = mo.expert_combine_grad(dout, y, r.plan, r.gates)
    dl = mo.route_grad(dgates, logits, r)
    # the loss sum(dout out) along a change of the logits that moves no choice
    top = torch.sort(logits, dim=1, descending=True).values
    step = float((top[:, 1] - top[:, 2]).min()) / 8
    assert step > 0
    d = torch.randn(200, 6, generator=g).cuda().clamp(-1, 1)

    def loss(l):
        q = mo.route(l, 2, normalize=True)
        assert torch.equal(q.experts, r.experts)
        return float((mo.expert_combine(y, q.plan, q.gates).double() * dout.double()).sum())
    step = min(step, 1e-3)
    diff = (loss(logits + step * d) - loss(logits - step * d)) / (2 * step)
    slope = float((dl.double() * d.double()).sum())
    # gates' rounding (2^-20 each, see the routing tests) over the step, and step^2 of the third derivative,
    # which is at most 1 for a softmax of two, both on the sum of |dout y|
    size = float((dout.double().abs() @ torch.ones(40, 1).cuda().double()).sum()) * float(y.abs().max())
    assert abs(diff - slope) <= size * (2.0 ** -20 / step + step * step)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_captured_layer_replays_on_new_inputs(dtype):
    args = on_gpu(problem(20, tokens=600), dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(*args, 5)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(*args, 5)
    for seed in (21, 22, 23, 20):
        fresh = on_gpu(problem(seed, tokens=600), dtype)
        for a, b in zip(args, fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("out", "dtable", "dw1", "dw2", "dgates"), held, layer(*fresh, 5)):
            assert torch.equal(a, b), (seed, name)


def test_two_graphs_that_share_nothing_replay_in_turn():
    graphs, inputs = [], []                                   # a graph reads the memory of its inputs
    for seed in (30, 31):
        x = torch.randn(700, 40, generator=torch.Generator().manual_seed(seed)).cuda()
        w = torch.randn(8, 24, 40, generator=torch.Generator().manual_seed(seed + 9)).cuda()

        inputs += [x, w]

        def run(x=x, w=w):
            r = mo.route(x[:, :8], 3)
            y = mo.expert_linear(x, w, r.plan, gather=True)
            return mo.expert_combine(y, r.plan, r.gates), mo.embedding_grad(y, r.plan.tokens, 700)
        want = run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        graphs.append((graph, got, want))
    for _ in range(3):
        for graph, got, want in graphs + graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_repeat_bit_for_bit():
    g = torch.Generator().manual_seed(40)
    x, w = torch.randn(3000, 72, generator=g).cuda(), torch.randn(12, 56, 72, generator=g).cuda()
    ids, dy = torch.randint(0, 50, (3000,), generator=g).cuda(), torch.randn(3000, 56, generator=g).cuda()

    def run():
        r = mo.route(x[:, :12], 2)
        y = mo.expert_linear(x, w, r.plan, gather=True)
        out = mo.expert_combine(y, r.plan, r.gates)
        dyr, dg = mo.expert_combine_grad(dy, y, r.plan, r.gates)
        return (r.gates, r.plan.tokens, y, out, dyr, dg, *mo.expert_linear_grad(dyr, w, x, r.plan, gather=True),
                mo.embedding_grad(dy, ids, 50))
    first = run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_calls_on_other_streams_and_from_threads():
    """Each thread with a stream of its own, all at once."""
    args = [on_gpu(problem(50 + i, tokens=400), F32) for i in range(4)]
    want = [layer(*a, 5) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(8):
                    got = layer(*args[i], 5)
                s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)
        except Exception as e:   # noqa: BLE001 (a thread's failure is the test's)
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_plans_that_were_written_over_are_not_followed():
    """Indexes of no row or token: nothing is read or written outside the tensors."""
    g = torch.Generator().manual_seed(60)
    x, w = torch.randn(50, 16, generator=g).cuda(), torch.randn(4, 24, 16, generator=g).cuda()
    plan = mo.expert_plan(torch.randint(0, 4, (50, 2), generator=g).cuda(), 4)
    plan.tokens[:7] = torch.tensor([50, -3, 1 << 30, -(1 << 31), 51, -1, (1 << 31) - 1], dtype=torch.int32)
    plan.place[1] = torch.tensor([100, -5], dtype=torch.int32)
    room = torch.full((102, 24), 7.0, device="cuda")
    y = mo.expert_linear(x, w, plan, gather=True, out=room[1:101])
    assert not y[:7].any() and (room[0] == 7).all() and (room[101] == 7).all()     # no token: a row of zeros
    out = mo.expert_combine(y, plan)
    assert not out[1].any() and torch.isfinite(out).all()
    _, dw = mo.expert_linear_grad(y, None, x, plan, gather=True)
    assert torch.isfinite(dw).all()
    plan.offsets.copy_(torch.tensor([-5, 300, 20, 1 << 30, 60], dtype=torch.int32))
    room.fill_(7.0)
    mo.expert_linear(x, w, plan, gather=True, out=room[1:101])
    _, dw = mo.expert_linear_grad(torch.ones(100, 24, device="cuda"), None, x, plan, gather=True)
    torch.cuda.synchronize()
    assert (room[0] == 7).all() and (room[101] == 7).all() and torch.isfinite(dw).all()
