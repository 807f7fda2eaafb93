"""Calls of the 4-bit operators that the documentation allows and that are easy
to get wrong: slices of one buffer, tensors without features, factors, seeds,
gradients beside autograd."""
import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from oracle import mx_oracle as mx
from tests.gpu_helpers import announce, host

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def _rand(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(dtype).cuda()


def test_outputs_that_are_slices_of_one_buffer():
    """A single row, a column slice and every second row of one buffer share nothing."""
    announce("one buffer's slices as outputs")
    xs = [mo.mx_quantize(_rand(r, 64, BF16, r)) for r in (1, 17, 9)]
    w = mo.mx_quantize(_rand(30, 64, BF16, 40))
    buf = torch.full((18, 100), 7.0, device="cuda")
    outs = [buf[1:2, :30], buf[:17, 30:60], buf[::2, 60:90]]
    mo.mx_matmul(xs, [w] * 3, out=outs)
    for o, x in zip(outs, xs):
        assert torch.equal(o, mo.mx_matmul(x, w, dtype=F32))
    assert bool((buf[0, :30] == 7.0).all() and (buf[2:, :30] == 7.0).all() and (buf[1::2, 60:] == 7.0).all())
    with pytest.raises(mo._lib.MuonError):
        mo.mx_matmul(xs, [w] * 3, out=[buf[1:2, 1:31], buf[:17, 30:60], buf[::2, 60:90]])
    x = _rand(17, 60, BF16, 3)
    wide = torch.zeros(17, 120, dtype=BF16, device="cuda")
    wide[:, :60] = x
    mo.dropout(wide[4:5, :60], 0.3, 9, out=wide[4:5, 60:])
    assert torch.equal(wide[4:5, 60:], mo.dropout(x[4:5], 0.3, 9)) and torch.equal(wide[:, :60], x)


@pytest.mark.parametrize("lead", [(), (6,), (2, 3), (2, 10), (0, 3)])
def test_layers_without_features(lead):
    """No inputs give zeros, no outputs give no gradient; leading dimensions stay."""
    announce(f"layers without features {lead}")
    n = int(np.prod(lead, dtype=np.int64))
    none, some = torch.zeros(5, 0, device="cuda", dtype=BF16), torch.zeros(0, 5, device="cuda", dtype=BF16)
    x = torch.zeros(*lead, 0, device="cuda", dtype=BF16)
    pair = mo.mx_quantize(none, "both")
    y = mo.mx_linear(x, pair.w)
    assert tuple(y.shape) == (*lead, 5) and not y.any()
    y, saved = mo.mx_linear(x, pair.w, save=True)
    assert tuple(y.shape) == (*lead, 5) and not y.any()
    dx, dw = mo.mx_linear_grad(torch.ones_like(y), pair.w_t, saved)
    assert tuple(dx.shape) == (*lead, 0) and tuple(dw.shape) == (5, 0)
    assert tuple(mo.dropout(x, 0.5, 3).shape) == (*lead, 0)
    # and a layer without outputs
    x = torch.ones(*lead, 5, device="cuda", dtype=BF16)
    pair = mo.mx_quantize(some, "both")
    y, saved = mo.mx_linear(x, pair.w, save=True)
    assert tuple(y.shape) == (*lead, 0)
    dx, dw = mo.mx_linear_grad(y, pair.w_t, saved)
    assert tuple(dx.shape) == (*lead, 5) and not dx.any() and tuple(dw.shape) == (0, 5)
    assert saved.x_t.cols == (n if lead else 1)


@pytest.mark.parametrize("shape", [(), (1,)])
def test_a_seed_advanced_between_forward_and_backward(shape):
    """The gradient has the forward pass's mask, eagerly and in a replayed graph."""
    announce(f"advanced seed {shape}")
    w, x, dy = _rand(40, 64, BF16, 1), _rand(33, 64, BF16, 2), _rand(33, 40, BF16, 3)
    pair = mo.mx_quantize(w, "both")

    def step(seed, advance=False):
        y, saved = mo.mx_linear(x, pair.w, save=True, dropout=0.4, dropout_seed=seed)
        if advance:
            seed += 1
        return (y, *mo.mx_linear_grad(dy, pair.w_t, saved, seed=11))
    seed = torch.full(shape, 5, dtype=torch.int64, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(step(seed, True), step(5)))
    assert int(seed) == 6
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(seed, True)
    for t in (6, 7, 8, -3):
        if t < 0:
            seed.fill_(t)
        g.replay()
        got = [o.clone() for o in out]
        (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step(t))), t
        assert int(seed) == t + 1
    for bad in (torch.zeros(1, dtype=torch.int64), torch.zeros(1, device="cuda"),
                torch.zeros(2, dtype=torch.int64, device="cuda")):
        with pytest.raises(ValueError):
            step(bad)


def test_layers_in_an_autograd_function():
    """The two passes as the halves of an autograd.Function, beside torch's own operations."""
    announce("autograd.Function")
    w = _rand(40, 64, BF16, 1)
    pair = mo.mx_quantize(w, "both")

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight):
            y, ctx.saved = mo.mx_linear(x, pair.w, save=True, dropout=0.2, dropout_seed=4)
            return y

        @staticmethod
        def backward(ctx, dy):
            return mo.mx_linear_grad(dy.contiguous(), pair.w_t, ctx.saved, seed=5)
    x = _rand(33, 64, F32, 2).requires_grad_()
    weight = w.float().requires_grad_()
    y = Layer.apply(x, weight)
    (y * y).sum().backward()
    with torch.no_grad():
        want, saved = mo.mx_linear(x, pair.w, save=True, dropout=0.2, dropout_seed=4)
        dx, dw = mo.mx_linear_grad(2 * want, pair.w_t, saved, seed=5)
    assert torch.equal(y, want) and torch.equal(x.grad, dx) and torch.equal(weight.grad, dw)
    for f in (lambda: mo.mx_linear(x, pair.w), lambda: mo.dropout(x, 0.1, 1),
              lambda: mo.mx_linear_grad(y, None, saved)):
        with pytest.raises(ValueError, match="autograd"):
            f()
    assert mo.mx_quantize(weight).shape == (40, 64)
    assert len(mo.Muon([torch.nn.Parameter(w.clone())], mx=True).mx) == 1


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (17, 129), (65, 200), (130, 257), (300, 5)])
def test_blocks_past_the_last_column_are_zeros_with_an_ordinary_scale(rows, cols):
    """What a product reads there adds nothing to a row, whatever the row holds."""
    announce(f"padding {rows}x{cols}")
    for dtype in (BF16, F32):
        x = _rand(rows, cols, dtype, 7)
        x[0, -1] = float("nan")
        x[-1, 0] = float("inf")
        for kw in (dict(), dict(seed=3), dict(dropout=0.4, dropout_seed=2), dict(seed=3, dropout=0.4, dropout_seed=2)):
            q, qt = mo.mx_quantize(x, "both", **kw)
            for m in (q, qt, mo.mx_quantize(x, False, **kw), mo.mx_quantize(x, True, **kw)):
                kt, rt, st = -(-m.cols // 128), -(-m.rows // 16), -(-m.rows // 64)
                raw = m.data.cpu().numpy()
                n = kt * rt * 1024
                # [k tile, row tile, block in k tile, row in tile, bytes]
                codes = raw[:n].reshape(kt, rt, 4, 16, 16)
                scales = raw[n:].reshape(kt, st, 4, 16, 4)
                for b in range(-(-m.cols // 32), 4 * kt):
                    for r in range(m.rows):
                        assert not codes[b // 4, r // 16, b % 4, r % 16].any()
                        assert scales[b // 4, r // 64, b % 4, r % 16, r % 64 // 16] != 255
                # and the elements past it in its own block
                last = -(-m.cols // 32) - 1
                for e in range(m.cols - 32 * last, 32):
                    byte = codes[last // 4, :, last % 4].reshape(rt * 16, 16)[:m.rows, e // 2]
                    assert not (byte >> (4 * (e & 1)) & 15).any()


def test_layers_of_a_shape_with_seeds_of_their_own():
    """The documented loop: seeds step * layers + layer give layers and steps
    masks and roundings of their own; one seed gives the same ones."""
    announce("seeds by layer")
    mats = [_rand(64, 96, BF16, 1), _rand(64, 96, BF16, 2)]
    opt = mo.Muon(mats, lr=0.02, mx=True)
    x, dy = torch.ones(50, 96, dtype=BF16, device="cuda"), _rand(50, 64, BF16, 4)
    masks, rounded = [], []
    for step in range(2):
        pairs = []
        for i in range(len(mats)):
            seed = step * len(mats) + i
            y, saved = mo.mx_linear(x, opt.mx[i].w, save=True, dropout=0.5, dropout_seed=seed)
            dx, pair = mo.mx_linear_grad(dy, opt.mx[i].w_t, saved, seed=seed, pair=True)
            masks.append(saved.x_t.dequantize(F32) != 0)
            rounded.append(pair[0].dequantize(F32))
            pairs.append(pair)
        opt.step(pairs)
    for a in range(4):
        for b in range(a):
            assert not torch.equal(masks[a], masks[b]) and not torch.equal(rounded[a], rounded[b])
    again = mo.mx_linear(x, opt.mx[0].w, save=True, dropout=0.5, dropout_seed=3)[1]
    assert torch.equal(again.x_t.dequantize(F32) != 0, masks[3])
