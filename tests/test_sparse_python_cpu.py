"""Host-only checks of the expert layers' and the embedding's Python layer: what it
refuses and what it hands on.  The library's calls are replaced by a recorder."""
import struct

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
        muon_embedding_grad_workspace_bytes = staticmethod(lambda *a: 64)
    monkeypatch.setattr(experts, "_call", lambda name, dev, *a: seen.append((name, a)) or 0)
    monkeypatch.setattr(experts, "_gpu", lambda dev: dev)
    monkeypatch.setattr(_lib, "load", lambda: Library)
    return seen


def _plan(tokens=5, k=2, n=3):
    return experts.ExpertPlan(torch.zeros(2 * tokens * k + n + 1, dtype=torch.int32), tokens, k, n, CPU)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="GPU"):
        mo.route(torch.zeros(3, 4), 2)
    with pytest.raises(ValueError, match="GPU"):
        mo.expert_plan(torch.zeros(3, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="GPU"):
        mo.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 5))
    with pytest.raises(ValueError, match="GPU"):
        mo.embedding_grad(torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), 4)


def test_a_plans_arrays_and_descriptor():
    p = _plan(5, 2, 3)
    assert p.place.shape == (5, 2) and p.tokens.shape == (10,) and p.offsets.shape == (4,) and p.slots == 10
    o, t, q, n, k, e = struct.unpack("PPPqii", p.desc)
    assert (o, t, q) == (p.offsets.data_ptr(), p.tokens.data_ptr(), p.place.data_ptr()) and (n, k, e) == (5, 2, 3)
    ends = sorted((a.data_ptr(), a.data_ptr() + 4 * a.numel()) for a in (p.offsets, p.tokens, p.place))
    assert all(a[1] <= b[0] for a, b in zip(ends, ends[1:]))


def test_routing_shares_one_allocation_without_overlap(calls):
    r = mo.route(torch.zeros(5, 7), 3, normalize=1)
    (name, a), = calls
    assert name == "muon_route" and a[1] == 1 and a[2] == r.gates.data_ptr() and a[3] == r.experts.data_ptr()
    parts = (r.gates, r.experts, r.plan.offsets, r.plan.tokens, r.plan.place)
    ends = sorted((t.data_ptr(), t.data_ptr() + 4 * t.numel()) for t in parts)
    assert all(x[1] <= y[0] for x, y in zip(ends, ends[1:]))
    assert r.gates.dtype == F32 and r.gates.shape == r.experts.shape == (5, 3) and r.normalize is True
    mo.route_grad(torch.zeros(5, 3), torch.zeros(5, 7), r)
    assert calls[-1][0] == "muon_route_grad" and calls[-1][1][4:6] == (3, 1)


def test_argument_errors(calls):
    p, x, w, dy = _plan(), torch.zeros(10, 4), torch.zeros(3, 6, 4), torch.zeros(10, 6)
    bad = [
        lambda: mo.route(torch.zeros(4), 1), lambda: mo.route(torch.zeros(2, 4), 0), lambda: mo.route(torch.zeros(2, 4), 65),
        lambda: mo.route(torch.zeros(2, 513), 1), lambda: mo.route(torch.zeros(2, 4, dtype=torch.float16), 1),
        lambda: mo.route(torch.zeros(4, 2).t(), 1),
        lambda: mo.expert_plan(torch.zeros(4, dtype=torch.int32), 3), lambda: mo.expert_plan(torch.zeros(4, 2), 3),
        lambda: mo.expert_plan(torch.zeros(4, 2, dtype=torch.int32), 0),
        lambda: mo.expert_plan(torch.zeros(2, 4, dtype=torch.int32).t(), 3),
        lambda: mo.expert_linear(x, w, None), lambda: mo.expert_linear(x, w[0], p), lambda: mo.expert_linear(x[:5], w, p),
        lambda: mo.expert_linear(x, w, p, gather=True), lambda: mo.expert_linear(x[:, :3], w, p),
        lambda: mo.expert_linear(x, w[:2], p), lambda: mo.expert_linear(x, w.transpose(1, 2), p),
        lambda: mo.expert_linear(x, w[:1].expand(3, 6, 4), p), lambda: mo.expert_linear(x, w, p, out=torch.zeros(10, 5)),
        lambda: mo.expert_linear(x, w, p, dtype=torch.float16), lambda: mo.expert_linear(x.half(), w.half(), p),
        lambda: mo.expert_linear_grad(dy[:, :5], w, x, p), lambda: mo.expert_linear_grad(dy, w, x[:, :3], p),
        lambda: mo.expert_linear_grad(dy, w, None, p, out=torch.zeros(3, 6, 4)),
        lambda: mo.expert_linear_grad(dy, w, x, p, accumulate=True),
        lambda: mo.expert_linear_grad(dy, w, x, p, out=torch.zeros(3, 4, 6)),
        lambda: mo.expert_linear_grad(dy, w, x, p, grad_dtype=torch.float64),
        lambda: mo.expert_combine(x[:5], p), lambda: mo.expert_combine(x, p, torch.zeros(5, 3)),
        lambda: mo.expert_combine(x, p, torch.zeros(5, 2, dtype=BF16)), lambda: mo.expert_combine(x, p, torch.zeros(2, 5).t()),
        lambda: mo.expert_combine(x, p, out=torch.zeros(4, 4)),
        lambda: mo.expert_combine_grad(torch.zeros(5, 3), x, p, torch.zeros(5, 2)),
        lambda: mo.expert_combine_grad(torch.zeros(5, 4), x, p, None), lambda: mo.expert_gather(x, p),
        lambda: mo.route_grad(torch.zeros(5, 2), torch.zeros(5, 4), mo.Routing(torch.zeros(5, 2), torch.zeros(5, 2), p, False)),
        lambda: mo.embedding(torch.zeros(3), torch.zeros(4, 5)), lambda: mo.embedding(torch.zeros(3, dtype=torch.int16), torch.zeros(4, 5)),
        lambda: mo.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(5)),
        lambda: mo.embedding(torch.zeros(4, 3, dtype=torch.int64).t(), torch.zeros(4, 5)),
        lambda: mo.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 5), out=torch.zeros(3, 4)),
        lambda: mo.embedding_grad(torch.zeros(4, 5), torch.zeros(3, dtype=torch.int64), 4),
        lambda: mo.embedding_grad(torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), 4, accumulate=True),
        lambda: mo.embedding_grad(torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), 4, out=torch.zeros(5, 5)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    assert not calls


def test_tensors_whose_gradient_would_be_lost_are_refused(calls):
    p, x, w = _plan(), torch.zeros(10, 4), torch.zeros(3, 6, 4)
    ids, gates = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 2)

    def needs(t):
        return t.clone().requires_grad_(True)
    lost = [lambda: mo.route(needs(torch.zeros(2, 4)), 1), lambda: mo.expert_linear(needs(x), w, p),
            lambda: mo.expert_linear(x, needs(w), p), lambda: mo.expert_combine(needs(x), p),
            lambda: mo.expert_combine(x, p, needs(gates)), lambda: mo.expert_gather(needs(x[:5]), p),
            lambda: mo.embedding(ids, needs(torch.zeros(4, 5)))]
    for f in lost:
        with pytest.raises(ValueError, match="autograd"):
            f()
    assert not calls
    with torch.no_grad():
        for f in lost:
            f()
    assert len(calls) == len(lost)


def test_long_gathered_rows_are_sorted_first(calls):
    """Rows that span more than a product addresses, of tensors that share one row's memory."""
    tokens = 1 << 20
    p = experts.ExpertPlan(torch.zeros(2 * tokens + 4, dtype=torch.int32), tokens, 1, 3, CPU)
    row = torch.zeros(8, dtype=BF16)
    x = row.as_strided((tokens, 8), (0, 1))
    experts_mat, experts._mat = experts._mat, lambda t, dev: (t.data_ptr(), *t.shape, 2048, 0, 0)
    try:
        class Far(torch.Tensor):
            def stride(self, *a):
                return 2048 if a == (0,) else (2048, 1)
        mo.expert_linear(x.as_subclass(Far), torch.zeros(3, 4, 8, dtype=BF16), p, gather=True)
    finally:
        experts._mat = experts_mat
    assert [c[0] for c in calls] == ["muon_expert_gather", "muon_expert_linear"]
    assert calls[1][1][3] == 0


def test_versions_of_given_outputs_rise(calls):
    p, x, w = _plan(), torch.zeros(10, 4), torch.zeros(3, 6, 4)
    out, dw, table = torch.zeros(10, 6), torch.zeros(3, 6, 4), torch.zeros(4, 5)
    mo.expert_linear(x, w, p, out=out)
    mo.expert_linear_grad(torch.zeros(10, 6), None, x, p, out=dw)
    mo.embedding_grad(torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), 4, out=table, accumulate=True)
    assert out._version == dw._version == table._version == 1
