"""Pins of the float64 oracle of routing, expert layers and embedding: values worked
by hand, torch's own gradients in float64, and sums that have to agree."""
import math

import numpy as np
import pytest
import torch

from oracle import sparse_oracle as so


def test_plan_by_hand():
    choice = np.array([[2, 0], [0, 3], [-1, 2], [0, 0]])      # 3 and -1 are no experts of three
    offsets, tokens, place = so.plan(choice, 3)
    assert offsets.tolist() == [0, 4, 4, 6]
    assert tokens.tolist() == [0, 1, 3, 3, 0, 2, -1, -1]
    assert place.tolist() == [[4, 0], [1, -1], [-1, 5], [2, 3]]


def test_route_by_hand():
    l = np.array([[0.0, math.log(2), 0.0, math.log(4)], [1.0, -math.inf, -math.inf, -math.inf], [-math.inf] * 4])
    gates, chosen = so.route(l, 3, False)
    assert chosen.tolist() == [[3, 1, 0], [0, -1, -1], [-1, -1, -1]]
    assert np.allclose(gates, [[4 / 8, 2 / 8, 1 / 8], [1, 0, 0], [0, 0, 0]], rtol=1e-15)
    gates, _ = so.route(l, 3, True)
    assert np.allclose(gates, [[4 / 7, 2 / 7, 1 / 7], [1, 0, 0], [0, 0, 0]], rtol=1e-15)
    gates, chosen = so.route(np.array([[1.0, math.nan, math.inf]]), 2, False)
    assert chosen.tolist() == [[1, 2]] and np.isnan(gates).all()


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_is_torchs(normalize):
    g = torch.Generator().manual_seed(1)
    l = torch.randn(7, 9, generator=g, dtype=torch.float64, requires_grad=True)
    dg = torch.randn(7, 3, generator=g, dtype=torch.float64)
    top, index = torch.topk(l, 3, dim=1)
    gates = torch.softmax(top, 1) if normalize else torch.softmax(l, 1).gather(1, index)
    gates.backward(dg)
    og, chosen = so.route(l.detach().numpy(), 3, normalize)
    assert np.array_equal(chosen, index.numpy()) and np.allclose(og, gates.detach().numpy(), rtol=1e-14)
    got = so.route_grad(dg.numpy(), l.detach().numpy(), og, chosen, normalize)
    assert np.abs(got - l.grad.numpy()).max() < 1e-15


def test_a_layer_and_its_gradients_are_torchs():
    g = torch.Generator().manual_seed(2)
    tokens, k, experts, cols, outs = 11, 2, 4, 5, 3
    choice = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)])
    x = torch.randn(tokens, cols, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(experts, outs, cols, generator=g, dtype=torch.float64, requires_grad=True)
    gates = torch.rand(tokens, k, generator=g, dtype=torch.float64, requires_grad=True)
    dout = torch.randn(tokens, outs, generator=g, dtype=torch.float64)
    out = torch.stack([sum(gates[t, j] * (w[choice[t, j]] @ x[t]) for j in range(k)) for t in range(tokens)])
    out.backward(dout)
    offsets, tk, place = so.plan(choice.numpy(), experts)
    xs, ws, gs = so.rows_of(x.detach().numpy(), tk), w.detach().numpy(), gates.detach().numpy()
    y = so.linear(xs, ws, offsets)
    assert np.allclose(so.combine(y, gs, place), out.detach().numpy(), rtol=1e-13)
    dy, dgates = so.combine_grad(dout.numpy(), y, gs, place)
    dx, dw = so.linear_grad(dy, ws, xs, offsets)
    assert np.allclose(dgates, gates.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(so.combine(dx, np.ones_like(gs), place), x.grad.numpy(), rtol=1e-12, atol=1e-14)


def test_embedding_and_gradient_are_torchs():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(6, 4, generator=g, dtype=torch.float64, requires_grad=True)
    ids, dy = torch.tensor([3, 0, 3, 5, -1, 6]), torch.randn(6, 4, generator=g, dtype=torch.float64)
    y = 0.5 * torch.nn.functional.embedding(ids[:4], w)
    y.backward(dy[:4])
    got = so.embedding(ids.numpy(), w.detach().numpy(), 0.5)
    assert np.allclose(got[:4], y.detach().numpy(), rtol=1e-15) and not got[4:].any()
    assert np.allclose(so.embedding_grad(dy.numpy(), ids.numpy(), 6, 0.5), w.grad.numpy(), rtol=1e-14)
