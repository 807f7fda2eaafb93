"""Host-only checks of the 4-bit operators' Python layer: what it keeps alive,
refuses and hands on.  The library's calls are replaced by recorders where a
check goes past the arguments."""
import gc
import weakref

import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import _lib, mx

CPU = torch.device("cpu")


def _held(rows, cols):
    """An MX4 in host memory."""
    return mx._new_mx([rows], [cols], CPU)[0]


def test_a_repeated_quantisation_keeps_the_memory_it_writes(monkeypatch):
    """The optimizer's list of 4-bit copies is the user's to change: what the
    packed descriptors point to must not be freed with it."""
    monkeypatch.setattr(mx, "_call", lambda *a: 0)
    pairs = [mx.MXPair(_held(8, 40), _held(40, 8))]
    memory = [weakref.ref(m.buffer) for m in pairs[0]]
    again = mx.quantize_again([torch.zeros(8, 40)], pairs)
    pairs.clear()
    gc.collect()
    assert all(m() is not None for m in memory)
    again()
    del again
    gc.collect()
    assert all(m() is None for m in memory)


def test_a_refused_workspace_is_an_error(monkeypatch):
    """A product whose second call, with a workspace, is refused too has no
    result to return."""
    seen = []

    def refused(*args):
        seen.append(args[-2])       # workspace bytes
        return _lib.CODES["MUON_E_WORKSPACE"]

    class Library:
        @staticmethod
        def muon_mx_matmul_workspace_bytes(*args):
            return 0                # as after a failed allocation on the host

    monkeypatch.setitem(mx._functions, "muon_mx_matmul", refused)
    monkeypatch.setattr(mx, "_current_device", lambda: None)
    monkeypatch.setattr(mx, "_current_stream", lambda i: None)
    monkeypatch.setattr(_lib, "load", lambda: Library)
    with pytest.raises(_lib.MuonError):
        mo.mx_matmul(_held(8, 40), _held(5, 40))
    assert seen == [0, 0]


@pytest.mark.parametrize("rows,few", [((1 << 29) - 64, True), ((1 << 29) - 63, False)])
def test_a_layer_past_the_few_rows_grid_takes_the_general_product(monkeypatch, rows, few):
    w = mx.MX4(torch.empty(0, dtype=torch.uint8), 0, CPU, (0, 0, rows, 32))
    calls = []

    def record(name, dev, *args):
        calls.append(name)
        return 0
    monkeypatch.setattr(mx, "_call", record)
    monkeypatch.setattr(mx, "_gpu", lambda dev: dev)
    monkeypatch.setattr(mx, "_new_one", lambda r, c, dt, dev: (torch.empty(0), b""))
    mo.mx_linear(torch.zeros(2, 32), w)
    assert calls == (["muon_mx_matmul_rows"] if few else ["muon_mx_quantize", "muon_mx_matmul"])


@pytest.mark.parametrize("shape,rows", [((2, 3, 0), 6), ((0, 3, 4), 0), ((2, 0, 0), 0), ((0,), 1), ((7,), 1),
                                        ((2, 3, 4), 6)])
def test_rows_of_tensors_without_features(shape, rows):
    assert tuple(mx._rows_of(torch.zeros(shape)).shape) == (rows, shape[-1])


@pytest.mark.parametrize("kw", [dict(out=torch.zeros(4, 40)), dict(accumulate=True), dict(grad_dtype=torch.bfloat16),
                                dict(out=torch.zeros(4, 40), accumulate=True)])
def test_factors_are_not_accumulated(kw):
    """With pair=True nothing is multiplied, so there is nothing to write or add."""
    saved = mx.MXSaved(_held(40, 8), 0.0, None)
    with pytest.raises(ValueError, match="pair"):
        mo.mx_linear_grad(torch.zeros(8, 4), None, saved, pair=True, **kw)


def test_the_forward_pass_keeps_the_seed_that_it_used(monkeypatch):
    """A program may advance its seed tensor between a layer's forward and
    backward pass: the gradient needs the mask of the forward pass."""
    used = []

    def quantize(x, transpose, dropout, dropout_seed):
        used.append(dropout_seed)
        return mx.MXPair(_held(8, 40), _held(40, 8))
    monkeypatch.setattr(mx, "mx_quantize", quantize)
    monkeypatch.setattr(mx, "mx_matmul", lambda a, b, dtype: torch.zeros(8, 4))
    seed = torch.tensor([5])
    _, saved = mo.mx_linear(torch.zeros(8, 40), _held(4, 40), save=True, dropout=0.5, dropout_seed=seed)
    seed += 1
    assert int(saved.dropout_seed) == 5 and used[0] is saved.dropout_seed
    for given in (7, None):
        _, saved = mo.mx_linear(torch.zeros(8, 40), _held(4, 40), save=True, dropout=0.0, dropout_seed=given)
        assert saved.dropout_seed is given


def test_a_result_that_autograd_would_lose_is_refused(monkeypatch):
    """The operators record no graph: a tensor that requires a gradient is taken
    only where autograd does not record."""
    x = torch.zeros(2, 40, requires_grad=True)
    w, saved = _held(4, 40), mx.MXSaved(_held(40, 8), 0.0, None)
    dy = torch.zeros(8, 4, requires_grad=True)
    calls = (lambda: mo.mx_linear(x, w), lambda: mo.mx_linear(x, w, save=True), lambda: mo.dropout(x, 0.5, 1),
             lambda: mo.mx_linear_grad(dy, None, saved), lambda: mo.dropout(x[0], 0.5, 1))
    for f in calls:
        with pytest.raises(ValueError, match="autograd"):
            f()
    # where nothing is recorded the next refusal is that of host memory, and
    # weights are quantised whether they require gradients or not
    for f in calls:
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(ValueError, match="GPU"):
        mo.mx_quantize(x)


def test_results_written_into_given_tensors_count_as_changes(monkeypatch):
    """autograd refuses to use a saved tensor that was overwritten: it learns of
    that by the tensor's version."""
    monkeypatch.setattr(mx, "_call", lambda *a: 0)
    monkeypatch.setattr(mx, "_gpu", lambda dev: dev)
    big, q, w = torch.zeros(9, 60), _held(8, 40), _held(5, 40)
    saved = mx.MXSaved(_held(40, 8), 0.0, None)
    views = [big[:8, :5], big[:8, 10:15]]
    for write, t in ((lambda: mo.mx_matmul(q, w, out=big[:8, :5]), big),
                     (lambda: mo.mx_matmul([q, q], [w, w], out=views, accumulate=True), big),
                     (lambda: mo.mx_dequantize(q, out=big[:8, :40]), big),
                     (lambda: mo.mx_dequantize([q, q], out=[big[:8, :40], torch.zeros(8, 40)]), big),
                     (lambda: mo.dropout(big, 0.5, 1, out=big), big),
                     (lambda: mo.mx_linear_grad(torch.zeros(8, 5), None, saved, out=big[:5, :40]), big)):
        before = t._version
        write()
        assert t._version > before
    # the error that this gives
    p = torch.ones(8, 40, requires_grad=True)
    kept = p.detach().clone()
    loss = (p * kept).sum()
    mo.dropout(kept, 0.5, 1, out=kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # tensors of inference mode have no version
    with torch.inference_mode():
        t = torch.zeros(8, 5)
        mo.mx_matmul(q, w, out=t)
    mo.mx_matmul([q, q], [w, w], out=[t, big[:8, :5]])


def test_a_tangent_that_autograd_would_lose_is_refused():
    """Forward mode's derivatives would be lost as those of backward mode are."""
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        x, dy = (fw.make_dual(torch.zeros(n, c), torch.ones(n, c)) for n, c in ((2, 40), (8, 4)))
        w, saved = _held(4, 40), mx.MXSaved(_held(40, 8), 0.0, None)
        for f in (lambda: mo.mx_linear(x, w), lambda: mo.dropout(x, 0.5, 1), lambda: mo.mx_linear_grad(dy, None, saved)):
            with torch.no_grad(), pytest.raises(ValueError, match="autograd"):
                f()
        with pytest.raises(ValueError, match="GPU"):          # without a tangent the next refusal is that of host memory
            mo.mx_linear(fw.unpack_dual(x).primal, w)
