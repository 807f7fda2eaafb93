"""Arguments that the expert layers and the embedding refuse, one wrong at a time, and
what they take: host-only, the library's calls replaced by a recorder."""
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import _lib, experts

CPU = torch.device("cpu")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """Records the calls; the tensors stay in host memory."""
    seen = []

    class Library:
        muon_expert_plan_workspace_bytes = staticmethod(lambda *a: 0)
        muon_expert_linear_dw_workspace_bytes = staticmethod(lambda *a: 0)
        muon_embedding_grad_workspace_bytes = staticmethod(lambda *a: 0)
    monkeypatch.setattr(experts, "_call", lambda name, dev, *a: seen.append((name, a)) or 0)
    monkeypatch.setattr(experts, "_gpu", lambda dev: dev)
    monkeypatch.setattr(_lib, "load", lambda: Library)
    return seen


def _plan(tokens=5, k=2, n=3):
    return experts.ExpertPlan(torch.zeros(2 * tokens * k + n + 1, dtype=torch.int32), tokens, k, n, CPU)


@pytest.mark.parametrize("bad", [
    torch.zeros(5, 2, dtype=torch.int64),                     # topk's indexes
    torch.zeros(5, 2), torch.zeros(5, 2, dtype=torch.int16),
    torch.zeros(1, dtype=torch.int32), torch.zeros(5, 1, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32),
    torch.zeros(10, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32).t(),
    torch.zeros(5, 4, dtype=torch.int32)[:, ::2], torch.zeros(5, 2, dtype=torch.int32, device="meta"),
    [[0, 1]] * 5, None])
def test_route_grad_checks_a_routings_experts(calls, bad):
    """A routing is a tuple that a caller can make; its experts are read as dense int32."""
    good = mo.Routing(torch.zeros(5, 2), torch.zeros(5, 2, dtype=torch.int32), _plan(), False)
    with pytest.raises(ValueError, match="routing.experts"):
        mo.route_grad(torch.zeros(5, 2), torch.zeros(5, 3), good._replace(experts=bad))
    assert not calls
    mo.route_grad(torch.zeros(5, 2), torch.zeros(5, 3), good)
    assert [c[0] for c in calls] == ["muon_route_grad"]


def test_route_grad_checks_a_routings_gates_and_sizes(calls):
    good = mo.Routing(torch.zeros(5, 2), torch.zeros(5, 2, dtype=torch.int32), _plan(), True)
    for bad in (dict(gates=torch.zeros(5, 2, dtype=torch.float64)), dict(gates=torch.zeros(2, 5).t()), dict(gates=None),
                dict(gates=torch.zeros(10)), dict(gates=torch.zeros(5, 3)), dict(plan=None), dict(plan=_plan(n=4)),
                dict(gates=torch.zeros(5, 65), experts=torch.zeros(5, 65, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mo.route_grad(torch.zeros(5, 2), torch.zeros(5, 3), good._replace(**bad))
    with pytest.raises(ValueError):
        mo.route_grad(torch.zeros(5, 2), torch.zeros(5, 3), None)
    assert not calls


def _gradient_calls(mark):
    """Every tensor whose derivative a call would lose, marked by `mark`, one at a time."""
    p, x, w, dy = _plan(), torch.zeros(10, 4), torch.zeros(3, 6, 4), torch.zeros(10, 6)
    t, gates, ids = torch.zeros(5, 4), torch.zeros(5, 2), torch.zeros(3, dtype=torch.int64)
    logits, rows = torch.zeros(5, 3), torch.zeros(3, 5)
    r = mo.Routing(gates, torch.zeros(5, 2, dtype=torch.int32), p, False)
    return [
        lambda: mo.route(mark(logits), 1), lambda: mo.route_grad(mark(gates), logits, r),
        lambda: mo.route_grad(gates, mark(logits), r), lambda: mo.route_grad(gates, logits, r._replace(gates=mark(gates))),
        lambda: mo.expert_gather(mark(t), p), lambda: mo.expert_gather(t, p, out=mark(x)),
        lambda: mo.expert_linear(mark(x), w, p), lambda: mo.expert_linear(x, mark(w), p),
        lambda: mo.expert_linear(x, w, p, out=mark(dy)),
        lambda: mo.expert_linear_grad(mark(dy), w, x, p), lambda: mo.expert_linear_grad(dy, mark(w), x, p),
        lambda: mo.expert_linear_grad(dy, mark(w), None, p), lambda: mo.expert_linear_grad(dy, w, mark(x), p),
        lambda: mo.expert_linear_grad(dy, w, x, p, out=mark(w)),
        lambda: mo.expert_combine(mark(x), p), lambda: mo.expert_combine(x, p, mark(gates)),
        lambda: mo.expert_combine(x, p, out=mark(t)),
        lambda: mo.expert_combine_grad(mark(t), x, p, gates), lambda: mo.expert_combine_grad(t, mark(x), p, gates),
        lambda: mo.expert_combine_grad(t, x, p, mark(gates)),
        lambda: mo.embedding(ids, mark(t)), lambda: mo.embedding(ids, t, out=mark(torch.zeros(3, 4))),
        lambda: mo.embedding_grad(mark(rows), ids, 4), lambda: mo.embedding_grad(rows, ids, 5, out=mark(torch.zeros(5, 5))),
    ]


def test_every_tensor_that_requires_a_gradient_is_refused(calls):
    """Where autograd records; elsewhere each is taken."""
    lost = _gradient_calls(lambda t: t.clone().requires_grad_(True))
    for i, f in enumerate(lost):
        with pytest.raises(ValueError, match="autograd") as e:
            f()
            pytest.fail(f"call {i} was taken")
        assert "4-bit" not in str(e.value)
    assert not calls
    with torch.no_grad():
        for f in lost:
            f()
    assert len(calls) >= len(lost)


def test_every_tensor_with_a_tangent_is_refused(calls):
    """Forward-mode derivatives would be lost too, also under no_grad; not within a Function's forward."""
    with torch.autograd.forward_ad.dual_level():
        lost = _gradient_calls(lambda t: torch.autograd.forward_ad.make_dual(t.clone(), torch.ones_like(t)))
        for i, f in enumerate(lost):
            for recorded in (True, False):
                with torch.set_grad_enabled(recorded), pytest.raises(ValueError, match="autograd"):
                    f()
                    pytest.fail(f"call {i} was taken")
        assert not calls
        for f in _gradient_calls(lambda t: t):
            f()

        class Combine(torch.autograd.Function):
            @staticmethod
            def forward(ctx, y):
                return mo.expert_combine(y, _plan())

            @staticmethod
            def jvp(ctx, dy):
                return mo.expert_combine(dy, _plan())
        y = torch.autograd.forward_ad.make_dual(torch.zeros(10, 4), torch.ones(10, 4))
        assert torch.autograd.forward_ad.unpack_dual(Combine.apply(y)).tangent.shape == (5, 4)


def test_ids_and_choices_of_any_row_pitch(calls):
    """A column slice of a batch of tokens, as a language model's inputs are: dense copies of its rows are read."""
    batch = torch.arange(12).reshape(3, 4)
    read = []

    def ids_of(packed):
        p, n, size, _ = experts._IDS.unpack(packed)
        import ctypes
        kind = ctypes.c_int64 if size == 8 else ctypes.c_int32
        read.append(list((kind * n).from_address(p)))
    experts_call = experts._call
    experts._call = lambda name, dev, *a: ids_of(a[1 if name == "muon_embedding_grad" else 0]) or 0
    try:
        for ids in (batch[:, :-1], batch[:, 1:], batch.int()[:, 1:3], batch[::2], batch.expand(2, 3, 4), batch[:, :1],
                    batch[0].expand(5, 4)):
            y = mo.embedding(ids, torch.zeros(20, 5))
            assert y.shape == (*ids.shape, 5) and read.pop() == ids.reshape(-1).tolist()
            mo.embedding_grad(torch.zeros(*ids.shape, 5), ids, 20)
            assert read.pop() == ids.reshape(-1).tolist()
        mo.expert_plan(batch[:, 1:3], 12)
        assert read.pop() == batch[:, 1:3].reshape(-1).tolist()
    finally:
        experts._call = experts_call
    for bad in (batch.t(), batch[:, ::2], batch[:, 1]):       # numbers that are apart, as in a matrix's rows
        with pytest.raises(ValueError, match="contiguous"):
            mo.embedding(bad, torch.zeros(20, 5))


def test_a_plan_made_by_hand_has_room_for_its_arrays(calls):
    """Its arrays' addresses go to the device as they are."""
    good = torch.zeros(2 * 10 + 4, dtype=torch.int32)
    for a in ((good[:-1], 5, 2, 3, CPU), (good.long(), 5, 2, 3, CPU), (good.float(), 5, 2, 3, CPU),
              (torch.zeros(48, dtype=torch.int32)[::2], 5, 2, 3, CPU), (good.reshape(2, 12), 5, 2, 3, CPU), (None, 5, 2, 3, CPU),
              (torch.zeros(30, dtype=torch.int32)[6:], 5, 2, 3, CPU),
              (good, 5, 2, 3, torch.device("meta")), (good, 5, 2, 4, CPU), (good, 6, 2, 3, CPU), (good, 5, 0, 3, CPU),
              (good, 5, 2, 0, CPU), (good, -5, 2, 3, CPU), (good, 5, 65, 3, CPU)):
        with pytest.raises(ValueError):
            experts.ExpertPlan(*a)
    plan = experts.ExpertPlan(good, 5, 2, 3, CPU)
    mo.expert_combine(torch.zeros(10, 4), plan)
    made = mo.expert_plan(torch.zeros(5, 2, dtype=torch.int64), 3)
    assert type(made) is experts.ExpertPlan and made.place.shape == (5, 2) and made.buffer.numel() == 24
    assert [c[0] for c in calls] == ["muon_expert_combine", "muon_expert_plan"]
