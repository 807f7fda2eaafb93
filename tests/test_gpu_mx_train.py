"""The 4-bit operators as a training program uses them together with the
optimizer: 4-bit weights kept by the step, gradients given as 4-bit factors,
whole training steps captured and replayed, streams, threads, and matrices
past 32-bit offsets."""
import threading

import numpy as np
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from oracle import mx_oracle as mx
from tests.gpu_helpers import announce, host
from workloads import gen

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def _params(shapes, seed, dtype=BF16):
    return [gen.torch_param_matrix(r, c, seed, i, torch.device("cuda"), dtype=dtype)
            for i, (r, c) in enumerate(shapes)]


def _same_mx(a, b):
    assert a.shape == b.shape and torch.equal(a.dequantize(F32), b.dequantize(F32))


def _eager_work():
    x = torch.randn(512, 512, device="cuda")
    (x @ x).sum()
    torch.cuda.synchronize()


SHAPES = [(96, 160), (160, 96), (200, 333), (64, 64)]


@pytest.mark.parametrize("kw", [dict(wd=0.1), dict(beta_slow=0.99, cautious=True, beta_ema=0.99, wd=0.1)])
def test_step_keeps_the_4bit_weights(kw):
    announce(f"Muon mx {sorted(kw)}")
    ps = _params(SHAPES, 3)
    ps[1] = ps[1].float()            # both element types in one optimizer
    twin = [p.clone() for p in ps]
    opt, ref = mo.Muon(ps, mx=True, **kw), mo.Muon(twin, **kw)
    held = [(q.w, q.w_t) for q in opt.mx]
    for t in range(3):
        for q, p in zip(opt.mx, ps):
            fresh = mo.mx_quantize(p, "both")
            _same_mx(q.w, fresh.w)
            _same_mx(q.w_t, fresh.w_t)
        grads = [gen.torch_grad_matrix(r, c, 3, t, i, torch.device("cuda"), rms=1e-3, dtype=BF16)
                 for i, (r, c) in enumerate(SHAPES)]
        opt.step(grads)
        ref.step(grads)
        assert all(torch.equal(a, b) for a, b in zip(ps, twin))
    assert all(q.w is a and q.w_t is b for q, (a, b) in zip(opt.mx, held))
    with torch.no_grad():
        ps[0].mul_(2)
    opt.mx_refresh()
    _same_mx(opt.mx[0].w, mo.mx_quantize(ps[0]))
    assert ref.mx is None


def _batch(T, seed):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, c, generator=g).to(BF16).cuda(), (torch.randn(T, r, generator=g) * 1e-3).to(BF16).cuda())
            for r, c in SHAPES]


def _pairs(opt, batch, seed):
    out = []
    for q, (x, dy) in zip(opt.mx, batch):
        _, saved = mo.mx_linear(x, q.w, save=True)
        out.append(mo.mx_linear_grad(dy, None, saved, seed=seed, pair=True)[1])
    return out


def test_step_multiplies_gradient_factors():
    announce("gradients as 4-bit factors")
    ps = _params(SHAPES, 5)
    twin = [p.clone() for p in ps]
    opt, ref = mo.Muon(ps, mx=True), mo.Muon(twin)
    for t in range(2):
        pairs = _pairs(opt, _batch(300, t), 77 + t)
        dense = [mo.mx_matmul(a, b, dtype=F32) for a, b in pairs]
        # factors and dense gradients may be mixed
        opt.step([pairs[0], dense[1], pairs[2], pairs[3]])
        ref.step(dense)
        assert all(torch.equal(a, b) for a, b in zip(ps, twin))
        assert all(torch.equal(a, b) for a, b in zip(opt.mom, ref.mom))
    with pytest.raises(ValueError):
        opt.step([pairs[1], *pairs[1:]])
    assert opt.step_count == 2


def test_captured_step_with_factors_and_4bit_weights():
    announce("captured step with factors")
    ps = _params(SHAPES, 6)
    twin = [p.clone() for p in ps]
    opt, ref = mo.Muon(ps, mx=True), mo.Muon(twin, mx=True)
    pairs = _pairs(opt, _batch(9000, 0), 5)     # long enough for split products
    mirror = [tuple(mo.MX4(m.buffer, m.offset, m.device, m.desc) for m in p) for p in pairs]
    g = opt.graph(pairs)
    for t in range(4):
        new = _pairs(opt, _batch(9000, t + 1), 100 + t)
        for (a, b), (c, d) in zip(pairs, new):
            a.data.copy_(c.data)
            b.data.copy_(d.data)
        g.replay()
        ref.step(mirror)
        _eager_work()
        assert all(torch.equal(a, b) for a, b in zip(ps, twin)), t
        for q, r in zip(opt.mx, ref.mx):
            _same_mx(q.w, r.w)
            _same_mx(q.w_t, r.w_t)
    assert opt.step_count == ref.step_count == 4


def test_training_step_captured_with_a_device_seed():
    """Forward, backward and weight gradients of two layers in one graph; the
    seeds are device numbers, so each replay rounds and drops anew."""
    announce("captured training step")
    w1, w2 = _params([(96, 64), (40, 96)], 8)
    q1, q2 = mo.mx_quantize(w1, "both"), mo.mx_quantize(w2, "both")
    x = torch.randn(50, 64, device="cuda").to(BF16)
    dy = torch.randn(50, 40, device="cuda").to(BF16)
    seed = torch.tensor([3], dtype=torch.int64, device="cuda")

    def step(seed):
        h, s1 = mo.mx_linear(x, q1.w, save=True, dropout=0.2, dropout_seed=seed)
        y, s2 = mo.mx_linear(h, q2.w, save=True)
        dh, g2 = mo.mx_linear_grad(dy, q2.w_t, s2, seed=seed)
        dx, g1 = mo.mx_linear_grad(dh, q1.w_t, s1, seed=seed)
        return y, dx, g1, g2, mo.dropout(dx, 0.5, seed)
    step(seed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(seed)
    seen = []
    for t in (3, 4, 5, -1):
        seed.fill_(t)
        x.copy_(torch.randn(50, 64, device="cuda").to(BF16))
        g.replay()
        got = [o.clone() for o in out]
        _eager_work()
        want = step(t)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), t
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_gradient_of_a_loss_through_two_layers():
    """dx and dw of two layers against the formulas in float64 on the values
    that the 4-bit operands stand for."""
    announce("two layers against float64")
    torch.manual_seed(0)
    w1, w2 = _params([(96, 64), (40, 96)], 9)
    q1, q2 = mo.mx_quantize(w1, "both"), mo.mx_quantize(w2, "both")
    x = torch.randn(50, 64).cuda()
    t = torch.randn(50, 40).cuda()
    h, s1 = mo.mx_linear(x, q1.w, save=True)
    y, s2 = mo.mx_linear(h, q2.w, save=True)
    dy = y - t                                    # of half the squared distance
    dh, g2 = mo.mx_linear_grad(dy, q2.w_t, s2)
    dx, g1 = mo.mx_linear_grad(dh, q1.w_t, s1)

    def check(got, a, b):
        a, b = a.astype(np.float64), b.astype(np.float64)
        k = a.shape[1]
        s = np.abs(a) @ np.abs(b).T
        assert np.all(np.abs(host(got) - a @ b.T) <= (k * 2.0 ** -23 + 2.0 ** -24) * s)
    check(h, mx.rounded(host(x)), mx.rounded(host(w1)))
    check(y, mx.rounded(host(h)), mx.rounded(host(w2)))
    check(dh, mx.rounded(host(dy)), mx.rounded(host(w2), transpose=True))
    check(g2, mx.rounded(host(dy), transpose=True), mx.rounded(host(h), transpose=True))
    check(dx, mx.rounded(host(dh)), mx.rounded(host(w1), transpose=True))
    check(g1, mx.rounded(host(dh), transpose=True), mx.rounded(host(x), transpose=True))


def test_streams_and_threads():
    """Calls on several streams at once, from several threads, each with its
    own data, give what they give alone; split products included."""
    announce("streams and threads")
    jobs = []
    for i in range(4):
        x = _params([(100 + i, 6000)], 20 + i)[0]
        w = _params([(130, 6000)], 30 + i)[0]
        jobs.append((x, w, mo.mx_matmul(mo.mx_quantize(x, seed=i), mo.mx_quantize(w), dtype=F32),
                     mo.dropout(x, 0.3, i)))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        x, w, want, dropped = jobs[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = mo.mx_matmul(mo.mx_quantize(x, seed=i), mo.mx_quantize(w), dtype=F32)
                d = mo.dropout(x, 0.3, i)
                s.synchronize()
                if not (torch.equal(got, want) and torch.equal(d, dropped)):
                    bad.append(i)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_few_rows_are_the_rows_of_a_longer_product():
    """At most 16 rows take the kernel that quantises on the way; within the
    product's bound it gives the rows of the quantised product."""
    announce("few rows")
    for K, N in ((64, 32), (100, 33), (2560, 70), (5000, 200), (300, 8200)):
        w = _params([(N, K)], 40)[0]
        q = mo.mx_quantize(w)
        wq = mx.rounded(host(w)) if N * K < 200000 else host(q.dequantize(F32)).astype(np.float64)
        for rows in (1, 3, 4, 5, 16):
            for dt in (BF16, F32):
                x = (torch.randn(rows, K, device="cuda") * torch.exp(torch.randn(rows, K, device="cuda"))).to(dt)
                if rows == 5:
                    x[2, K // 2] = float("nan")
                got = host(mo.mx_linear(x, q)).astype(np.float64)
                xq = mx.rounded(host(x))
                if rows == 5:
                    assert np.isnan(got[2]).all()
                    xq[2] = 0
                    got[2] = 0
                s = np.abs(xq) @ np.abs(wq).T
                ref = xq @ wq.T
                tol = K * 2.0 ** -23 * s
                tol = tol + (2.0 ** -8 if dt == BF16 else 2.0 ** -24) * (np.abs(ref) + tol)
                assert np.all(np.abs(got - ref) <= tol), (K, N, rows, dt)
        # rows of a wider tensor, not 16-byte aligned
        big = torch.randn(4, K + 7, device="cuda").to(BF16)
        assert torch.equal(mo.mx_linear(big[:, 3:K + 3], q), mo.mx_linear(big[:, 3:K + 3].contiguous(), q))


def test_refused_layouts():
    announce("refused layouts")
    x = torch.randn(32, 64, device="cuda")
    for bad in (x.t(), x[:, ::2], x[:1].expand(32, 64), x.half(), x.view(4, 8, 64).transpose(0, 1)):
        with pytest.raises(ValueError):
            mo.mx_quantize(bad)
    q = mo.mx_quantize(x)
    with pytest.raises(ValueError):
        mo.mx_linear(torch.randn(3, 63, device="cuda"), q)
    with pytest.raises(ValueError):
        mo.mx_matmul(q, q, accumulate=True)
    with pytest.raises(ValueError):
        mo.mx_quantize(x, dropout=0.5)
    with pytest.raises(ValueError):
        mo.mx_quantize(x, seed=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(mo._lib.MuonError):
        mo.dropout(x, 1.0, 3)
    with pytest.raises(mo._lib.MuonError):
        mo.mx_matmul([q, q], [q, q], out=[x[:, :32], x[:, 16:48]])


def test_matrices_past_32_bit_offsets():
    """A matrix of more than 2^33 elements: its codes pass 4 GiB, its input 16
    and a product's output rows lie past 2^32 bytes."""
    announce("past 32-bit offsets")
    rows, cols = (1 << 20) + 100, 8256
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    marks = [0, 5, 777_777, rows - 130, rows - 1]
    g = torch.Generator().manual_seed(2)
    part = torch.randn(len(marks), cols, generator=g).to(BF16)
    x[torch.tensor(marks).cuda()] = part.cuda()
    q = mo.mx_quantize(x)
    assert q.nbytes > 1 << 32
    w = torch.randn(20, cols, generator=g).to(BF16).cuda()
    qw = mo.mx_quantize(w)
    y = mo.mx_matmul(q, qw, dtype=F32)
    a, b = mx.rounded(host(part.cuda())), mx.rounded(host(w))
    s = np.abs(a) @ np.abs(b).T
    got = host(y[torch.tensor(marks).cuda()])
    assert np.all(np.abs(got - a @ b.T) <= (cols * 2.0 ** -23 + 2.0 ** -24) * s)
    assert int((y != 0).any(1).sum()) == len(marks)
    del y
    d = mo.dropout(x, 0.5, 3, out=x)
    want = mx.dropout(np.ones((1, 16)), 0.5, 3)     # the mask of the first row's first elements
    assert np.array_equal(host(d[0, :16]) != 0, want[0] != 0)
    v = mo.mx_dequantize(q, out=d)
    assert np.array_equal(host(v[torch.tensor(marks).cuda()]).astype(np.float64), a)
    assert int((v != 0).any(1).sum()) == len(marks)
    del q, d, v
    t = mo.mx_quantize(x, True)                     # x now holds the values read back
    assert t.shape == (cols, rows) and t.nbytes > 1 << 32
    z = mo.mx_matmul(t, t, dtype=F32)               # x^T x, over a million rows
    # every marked row but 0 and 5 is alone in its block of 32, where a column's
    # one element, 1 or 1.5 times a power of two, is 4 or 6 scales: held exactly
    tail = mx.rounded(np.concatenate([a[:1], np.zeros((4, cols)), a[1:2], np.zeros((26, cols))]), transpose=True)
    b = np.concatenate([tail.T, a[2:]])
    want, s = b[:, :300].T @ b, np.abs(b[:, :300]).T @ np.abs(b)
    assert np.all(np.abs(host(z[:300]) - want) <= (len(marks) * 2.0 ** -23 + 2.0 ** -24) * s)


def test_preparing_a_step_launches_no_product():
    announce("step_prepare with factors")
    ps = _params(SHAPES, 9)
    opt = mo.Muon(ps, mx=True)
    pairs = _pairs(opt, _batch(64, 1), 3)
    opt.step(pairs)
    for g in opt._pgrads.values():
        g.fill_(7.0)
    opt.step_prepare(pairs)
    torch.cuda.synchronize()
    assert all(bool((g == 7.0).all()) for g in opt._pgrads.values())
