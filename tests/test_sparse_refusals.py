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
