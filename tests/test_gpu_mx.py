"""4-bit operators and dropout on the GPU against the float64 oracle.

Quantisation, reading back and dropout are compared bit for bit.  A product
sums K terms that are exact in fp32, so with the sum of their magnitudes S
each element is within K 2^-23 S of the exact one whatever the order of the
additions and however each of them rounds (one unit), plus half a step of the
output's type (2^-24 for fp32, 2^-8 for bf16)."""
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


def _rand(rows, cols, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if spread:
        x = x * torch.exp(2 * torch.randn(rows, cols, generator=g))
    return x.to(dtype).cuda()


def _same(got: torch.Tensor, want: np.ndarray, dtype=None):
    g = host(got).astype(np.float64)
    assert g.shape == want.shape
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(g[ok], want[ok])


def _tol(a, b, dtype):
    k = a.shape[1]
    s = np.abs(a) @ np.abs(b).T
    ref = np.abs(a @ b.T)
    return k * 2.0 ** -23 * s + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * (ref + k * 2.0 ** -23 * s)


SHAPES = [(1, 1), (1, 32), (3, 33), (16, 128), (17, 129), (64, 31), (65, 200), (130, 257), (7, 640),
          (300, 5)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_values_and_storage(rows, cols, dtype):
    announce(f"quantize {rows}x{cols} {dtype}")
    x = _rand(rows, cols, dtype, 11)
    xh = host(x)
    for seed in (None, 0x1234567890ABCDEF):
        q, qt = mo.mx_quantize(x, "both", seed=seed)
        _same(q.dequantize(F32), mx.rounded(xh, seed))
        _same(qt.dequantize(F32), mx.rounded(xh, seed, transpose=True))
        for m, turn in ((q, False), (qt, True)):
            u = xh.T if turn else xh
            r8 = None if seed is None else mx.randoms(*u.shape, 8, mx.ROUND_T if turn else mx.ROUND, 0, seed)
            codes, scales, valid = mx.storage(*mx.quantize(u, r8))
            raw = m.data.cpu().numpy()
            assert np.array_equal(raw[:codes.size], codes.ravel())
            assert np.array_equal(raw[codes.size:][valid.ravel()], scales.ravel()[valid.ravel()])
            # blocks past the last column have an ordinary scale in every stored row
            assert not np.any((raw[codes.size:] == 255)[valid.ravel()])
        one = mo.mx_quantize(x, False, seed=seed)
        two = mo.mx_quantize(x, True, seed=seed)
        _same(one.dequantize(F32), mx.rounded(xh, seed))
        _same(two.dequantize(F32), mx.rounded(xh, seed, transpose=True))
        _same(q.dequantize(BF16), mx.rounded(xh, seed))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_ties_extremes_and_non_finite(dtype):
    announce(f"quantize special values {dtype}")
    x = torch.zeros(12, 64, dtype=F32)
    x[0, :16] = torch.tensor([6, -5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.75, 5.0, 4.5, 3.0, -0.0, 0.125, 0.5])
    x[1] = 0.0
    x[2, 0] = float("inf")
    x[3, 40] = float("nan")
    x[4, 7] = float("-inf")
    x[5, :4] = torch.tensor([3.38e38, -1e38, 1e37, 1e-30])
    x[6, :4] = torch.tensor([1e-45, 2e-44, -1e-40, 3e-39])
    x[7, :4] = torch.tensor([2.0 ** -126, 2.0 ** -128, -2.0 ** -127, 1.5 * 2.0 ** -127])
    x[8, :3] = torch.tensor([6.0 * 2.0 ** -127, 5.0 * 2.0 ** -127, 2.5 * 2.0 ** -127])
    x[9, :33] = torch.linspace(-7, 7, 33)
    x[10, :2] = torch.tensor([6.015625, 6.0])
    x[11] = torch.finfo(dtype).min
    x = x.to(dtype).cuda()
    xh = host(x)
    for seed in (None, 5):
        for turn in (False, True):
            want = mx.rounded(xh, seed, transpose=turn)
            with np.errstate(over="ignore"):
                want32 = want.astype(np.float32).astype(np.float64)   # the top of the range overflows
            q = mo.mx_quantize(x, turn, seed=seed)
            _same(q.dequantize(F32), want32)


def test_stochastic_rounding_follows_the_formula_on_a_grid():
    announce("stochastic rounding over a fine grid")
    x = torch.linspace(-6, 6, 64 * 1024).view(64, 1024)
    x[:, ::32] = 6.0
    for dtype in (F32, BF16):
        xd = x.to(dtype).cuda()
        for seed in (1, 2):
            _same(mo.mx_quantize(xd, seed=seed).dequantize(F32), mx.rounded(host(xd), seed))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_strides_lists_and_out(dtype):
    announce(f"quantize strides and lists {dtype}")
    big = _rand(70, 300, dtype, 3)
    views = [big[:, 3:200], big[1:, :17], big[::2, 8:136], big[:0, :], big[:5, :0], big[5:6, 1:2]]
    got = mo.mx_quantize(views, "both", seed=9)
    for i, (v, (a, b)) in enumerate(zip(views, got)):
        vh = host(v) if v.numel() else np.zeros(tuple(v.shape))
        assert a.shape == tuple(v.shape) and b.shape == tuple(v.shape)[::-1]
        _same(a.dequantize(F32), mx.rounded(vh, 9, index=i))
        _same(b.dequantize(F32), mx.rounded(vh, 9, transpose=True, index=i))
    again = mo.mx_quantize(views, "both", seed=10, out=got)
    assert again[0].w is got[0].w
    _same(got[0].w.dequantize(F32), mx.rounded(host(views[0]), 10))
    # many matrices: more than one launch
    many = [_rand(5 + i, 40, dtype, i) for i in range(90)]
    for i, (v, q) in enumerate(zip(many, mo.mx_quantize(many, seed=4))):
        _same(q.dequantize(F32), mx.rounded(host(v), 4, index=i))
    # strided output of the reading back leaves what is around it
    dst = torch.full((72, 310), 7.0, dtype=dtype, device="cuda")
    q = mo.mx_quantize(views[0])
    mo.mx_dequantize(q, out=dst[1:71, 5:202])
    w = np.full((72, 310), 7.0)
    w[1:71, 5:202] = mx.rounded(host(views[0]))
    if dtype == BF16:   # bf16 holds every 4-bit value of this range
        _same(dst, w)
    else:
        _same(dst, w)


def test_quantize_with_dropout_is_quantize_of_dropout():
    announce("quantize with dropout")
    for dtype in (BF16, F32):
        x = _rand(37, 203, dtype, 8)
        x[3, 4] = float("nan")
        x[5, 6] = float("inf")
        a = mo.mx_quantize(x, "both", dropout=0.3, dropout_seed=77)
        b = mo.mx_quantize(mo.dropout(x, 0.3, 77), "both")
        for u, v in zip(a, b):
            _same(u.dequantize(F32), host(v.dequantize(F32)).astype(np.float64))


PRODUCTS = [(1, 1, 1), (1, 40, 32), (5, 3, 1), (16, 16, 128), (17, 33, 129), (64, 128, 256), (130, 70, 300),
            (200, 257, 640), (3, 130, 1000), (128, 128, 2048), (257, 300, 77), (33, 513, 4000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul(M, N, K, dtype):
    announce(f"matmul {M}x{N}x{K} {dtype}")
    a, b = _rand(M, K, BF16, 1), _rand(N, K, F32, 2)
    ah, bh = mx.rounded(host(a)), mx.rounded(host(b))
    qa, qb = mo.mx_quantize(a), mo.mx_quantize(b)
    got = host(mo.mx_matmul(qa, qb, dtype=dtype)).astype(np.float64)
    assert np.all(np.abs(got - ah @ bh.T) <= _tol(ah, bh, dtype))
    # into a strided output, added to what is there; the surroundings stay
    base = _rand(M + 2, N + 5, dtype, 4, spread=False)
    out = base.clone()
    mo.mx_matmul(qa, qb, out=out[1:M + 1, 3:N + 3], accumulate=True)
    want = host(base).astype(np.float64)
    prod = ah @ bh.T
    tol = np.zeros_like(want)
    step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    inner = want[1:M + 1, 3:N + 3]
    # the product's own error, the fp32 sum's rounding, the output's
    err = K * 2.0 ** -23 * (np.abs(ah) @ np.abs(bh).T)
    tot = np.abs(inner + prod) + err
    tol[1:M + 1, 3:N + 3] = err + (step + 2.0 ** -24) * 1.01 * tot
    want[1:M + 1, 3:N + 3] = inner + prod
    assert np.all(np.abs(host(out).astype(np.float64) - want) <= tol)


def test_matmul_scales_over_the_whole_range_and_nan_rows():
    announce("matmul scale range and NaN")
    K = 256
    a = _rand(20, K, F32, 5, spread=False) * torch.exp2(torch.arange(20).float().cuda() * 6 - 60)[:, None]
    b = _rand(40, K, F32, 6, spread=False) * torch.exp2(torch.arange(40).float().cuda() - 20)[:, None]
    a[3, 100] = float("nan")
    b[7, 9] = float("inf")
    a[5] = 0
    ah, bh = mx.rounded(host(a)), mx.rounded(host(b))
    got = host(mo.mx_matmul(mo.mx_quantize(a), mo.mx_quantize(b), dtype=F32)).astype(np.float64)
    with np.errstate(invalid="ignore"):
        ref = ah @ bh.T
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.isnan(got[3]).all() and np.isnan(got[:, 7]).all() and np.isfinite(got[4, :7]).all()
    ok = np.isfinite(ref)
    az, bz = np.nan_to_num(ah), np.nan_to_num(bh)
    assert np.all(np.abs(got - ref)[ok] <= _tol(az, bz, F32)[ok])


def test_matmul_lists_ragged_and_empty():
    announce("matmul lists")
    shapes = [(0, 30, 64), (17, 30, 64), (1, 200, 300), (5, 6, 0), (140, 0, 32), (129, 131, 97)] + \
             [(3 + i, 20, 40 + i) for i in range(60)]
    xs = [_rand(m, k, BF16, 20 + i) for i, (m, n, k) in enumerate(shapes)]
    ws = [_rand(n, k, BF16, 900 + i) for i, (m, n, k) in enumerate(shapes)]
    qx, qw = mo.mx_quantize(xs), mo.mx_quantize(ws)
    outs = mo.mx_matmul(qx, qw, dtype=F32)
    for (m, n, k), x, w, o in zip(shapes, xs, ws, outs):
        assert tuple(o.shape) == (m, n)
        if m * n == 0:
            continue
        ah = mx.rounded(host(x)) if k else np.zeros((m, 0))
        bh = mx.rounded(host(w)) if k else np.zeros((n, 0))
        assert np.all(np.abs(host(o) - ah @ bh.T) <= _tol(ah, bh, F32))
    # one right operand shared by all products; outputs that are column slices of one tensor
    buf = torch.zeros(17, 90, device="cuda")
    parts = [buf[:, 30 * j:30 * j + 30] for j in range(3)]
    mo.mx_matmul([qx[1]] * 3, [qw[1]] * 3, out=parts)
    assert all(torch.equal(p, outs[1]) for p in parts)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (37, 333), (130, 512), (5, 2049)])
def test_dropout(rows, cols, dtype):
    announce(f"dropout {rows}x{cols} {dtype}")
    x = _rand(rows, cols, dtype, 2)
    x[0, 0] = float("nan")
    if cols > 1:
        x[-1, -1] = float("inf")
    for p in (0.0, 1e-6, 0.1, 0.5, 0.999):
        want = torch.from_numpy(mx.dropout(host(x), p, 99)).to(dtype)
        got = mo.dropout(x, p, 99)
        _same(got, host(want).astype(np.float64))
        pad = torch.zeros(rows, cols + 3, dtype=dtype, device="cuda")
        mo.dropout(x, p, 99, out=pad[:, 1:cols + 1])
        _same(pad[:, 1:cols + 1], host(want).astype(np.float64))
        assert not pad[:, 0].any() and not pad[:, cols + 1:].any()
    y = x.clone()
    mo.dropout(y, 0.5, 3, out=y)
    _same(y, host(mo.dropout(x, 0.5, 3)).astype(np.float64))
    assert mo.dropout(x[:0], 0.5, 3).shape == (0, cols)


def test_dropout_of_leading_dimensions_and_seed_tensor():
    announce("dropout shapes and seed tensor")
    x = _rand(24, 40, BF16, 1).view(2, 3, 4, 40)
    y = mo.dropout(x, 0.3, 5)
    assert y.shape == x.shape and torch.equal(y.view(24, 40), mo.dropout(x.view(24, 40), 0.3, 5))
    v = x.view(-1)
    assert torch.equal(mo.dropout(v, 0.3, 5), mo.dropout(v.view(1, -1), 0.3, 5).view(-1))
    big = (1 << 63) + 12345
    s = torch.tensor([big - (1 << 64)], dtype=torch.int64, device="cuda")
    assert torch.equal(mo.dropout(x, 0.3, s), mo.dropout(x, 0.3, big))


def _linear_case(T, K, N, dtype, seed):
    x, w, dy = _rand(T, K, dtype, seed, spread=False), _rand(N, K, BF16, seed + 1, spread=False) * 0.05, \
        _rand(T, N, dtype, seed + 2, spread=False) * 1e-3
    return x, w, dy


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,N,p", [(1, 64, 48, 0.0), (5, 33, 70, 0.2), (40, 200, 130, 0.1), (257, 129, 64, 0.0)])
def test_linear_and_gradients_against_the_formula(T, K, N, p, dtype):
    announce(f"linear {T}x{K}->{N} p={p} {dtype}")
    x, w, dy = _linear_case(T, K, N, dtype, 40)
    pair = mo.mx_quantize(w, "both")
    y, saved = mo.mx_linear(x, pair.w, save=True, dropout=p, dropout_seed=11)
    dx, dw = mo.mx_linear_grad(dy, pair.w_t, saved, seed=12)
    assert y.dtype == dtype and dx.dtype == dtype and dw.dtype == F32
    xd = host(mo.dropout(x, p, 11)) if p else host(x)
    xq, xtq = mx.rounded(xd), mx.rounded(xd, transpose=True)
    wq, wtq = mx.rounded(host(w)), mx.rounded(host(w), transpose=True)
    dq, dtq = mx.rounded(host(dy), 12), mx.rounded(host(dy), 12, transpose=True)
    assert np.all(np.abs(host(y) - xq @ wq.T) <= _tol(xq, wq, dtype))
    assert np.all(np.abs(host(dw) - dtq @ xtq.T) <= _tol(dtq, xtq, F32))
    scale = 1.0
    ref, tol = dq @ wtq.T, _tol(dq, wtq, dtype)
    if p:
        t = int(np.floor(p * 65536 + 0.5))
        keep = mx.randoms(T, K, 16, mx.DROP, 0, 11) >= t
        scale = 65536 / (65536 - t)
        ref = np.where(keep, ref * scale, 0)
        # the scale is an fp32 number and the product with it rounds: 2^-24 each
        tol = np.where(keep, tol * scale + 2.0 ** -23 * np.abs(ref), 0)
    assert np.all(np.abs(host(dx) - ref) <= tol)
    if not p:
        assert torch.equal(mo.mx_linear(x, pair.w), y)


def test_linear_gradient_against_differences():
    """With inputs, weights and output gradient that 4 bits hold exactly the
    layer is linear, so differences along any 4-bit direction are its gradient."""
    announce("linear gradient against differences")
    g = torch.Generator().manual_seed(1)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

    def pick(r, c):   # every block of either orientation holds a 6, so the scale stays 1
        v = grid[torch.randint(0, 8, (r, c), generator=g)] * (torch.randint(0, 2, (r, c), generator=g) * 2 - 1)
        v[::8, :] = 6.0
        v[:, ::8] = 6.0
        return v.cuda()
    T, K, N = 64, 96, 32
    x, w, dy = pick(T, K), pick(N, K), pick(T, N)
    pair = mo.mx_quantize(w, "both")
    y, saved = mo.mx_linear(x, pair.w, save=True)
    dx, dw = mo.mx_linear_grad(dy, pair.w_t, saved)

    def loss(xx, ww):
        return float((mo.mx_linear(xx, mo.mx_quantize(ww)).double() * dy.double()).sum())
    base = loss(x, w)
    for r, c in ((1, 3), (17, 50), (63, 95)):
        step = x.clone()
        step[r, c] = 6.0 if x[r, c] != 6.0 else -6.0
        assert loss(step, w) - base == float(dx[r, c]) * float(step[r, c] - x[r, c])
    for r, c in ((1, 3), (17, 50), (31, 95)):
        step = w.clone()
        step[r, c] = 6.0 if w[r, c] != 6.0 else -6.0
        assert loss(x, step) - base == float(dw[r, c]) * float(step[r, c] - w[r, c])


def test_linear_shapes_pairs_and_accumulation():
    announce("linear shapes, pairs, accumulation")
    x, w, dy = _linear_case(48, 96, 80, BF16, 50)
    pair = mo.mx_quantize(w, "both")
    y, saved = mo.mx_linear(x.view(4, 12, 96), pair.w, save=True)
    assert y.shape == (4, 12, 80) and torch.equal(y.view(48, 80), mo.mx_linear(x, pair.w))
    dx, dw = mo.mx_linear_grad(dy.view(4, 12, 80), pair.w_t, saved, seed=3)
    assert dx.shape == (4, 12, 96)
    none, (a, b) = mo.mx_linear_grad(dy, None, saved, seed=3, pair=True)
    assert none is None and torch.equal(mo.mx_matmul(a, b, dtype=F32), dw)
    acc = torch.ones(80, 96, device="cuda")
    _, got = mo.mx_linear_grad(dy, None, saved, seed=3, out=acc, accumulate=True)
    assert got is acc and torch.equal(acc, dw + 1)
    # no tokens
    y0, s0 = mo.mx_linear(x[:0], pair.w, save=True)
    dx0, dw0 = mo.mx_linear_grad(dy[:0], pair.w_t, s0)
    assert y0.shape == (0, 80) and dx0.shape == (0, 96) and not dw0.any()


def test_matmul_output_past_the_caches():
    """Outputs between half of the last cache and all of it take another kind of store."""
    M, N, K = 8200, 8200, 130
    announce(f"matmul {M}x{N}x{K} past the caches")
    qa, qb = mo.mx_quantize(_rand(M, K, BF16, 1)), mo.mx_quantize(_rand(N, K, BF16, 2))
    out = torch.full((M + 1, N + 3), 7.0, device="cuda", dtype=BF16)
    mo.mx_matmul(qa, qb, out=out[:M, :N])
    assert 128 << 20 < 2 * M * N <= 256 << 20
    rows = torch.tensor([0, 1, 127, 128, 255, 4095, 4096, 8191, 8192, M - 1], device="cuda")
    da, db = mo.mx_dequantize(qa, dtype=F32), mo.mx_dequantize(qb, dtype=F32)
    exact = da[rows].double() @ db.double().t().contiguous()
    size = da[rows].double().abs() @ db.double().abs().t().contiguous()
    tol = K * 2.0 ** -23 * size + 2.0 ** -8 * (exact.abs() + K * 2.0 ** -23 * size)
    assert bool(((out[rows, :N].double() - exact).abs() <= tol).all())
    assert bool((out[M:] == 7.0).all()) and bool((out[:, N:] == 7.0).all())


def test_numpy_arguments():
    """numpy's booleans and integers do what Python's do."""
    announce("numpy arguments")
    x = _rand(40, 70, BF16, 4)
    for yes in (1, np.True_):
        assert torch.equal(mo.mx_quantize(x, yes).dequantize(F32), mo.mx_quantize(x, True).dequantize(F32))
    for no in (0, np.False_):
        assert torch.equal(mo.mx_quantize(x, no).dequantize(F32), mo.mx_quantize(x).dequantize(F32))
    for seed in (np.int64(-5), np.uint64(2 ** 64 - 5)):
        assert torch.equal(mo.dropout(x, 0.3, seed), mo.dropout(x, 0.3, -5))
        assert torch.equal(mo.mx_quantize(x, seed=seed).dequantize(F32), mo.mx_quantize(x, seed=-5).dequantize(F32))


@pytest.mark.parametrize("M,N,K", [(256, 128, 64), (300, 264, 200), (513, 385, 130), (128, 128, 9000), (40, 70, 33)])
def test_matmul_with_dropout_is_dropout_of_matmul(M, N, K):
    """Whole tiles, edges and split contractions drop the elements that dropout()
    drops from the fp32 product, and scale them before the only rounding."""
    announce(f"matmul with dropout {M}x{N}x{K}")
    a, b = mo.mx_quantize(_rand(M, K, BF16, 31)), mo.mx_quantize(_rand(N, K, BF16, 32))
    want = mo.dropout(mo.mx_matmul(a, b, dtype=F32), 0.3, 99)
    assert torch.equal(mo.mx_matmul(a, b, dtype=F32, dropout=0.3, dropout_seed=99), want)
    assert torch.equal(mo.mx_matmul(a, b, dropout=0.3, dropout_seed=99), want.to(BF16))
    for dt in (F32, BF16):
        out = torch.full((M, N + 5), 3.0, device="cuda", dtype=dt)
        base = _rand(M, N, dt, 33)
        out[:, :N] = base
        mo.mx_matmul(a, b, out=out[:, :N], accumulate=True, dropout=0.3, dropout_seed=99)
        assert torch.equal(out[:, :N], (base.float() + want).to(dt))
        assert bool((out[:, N:] == 3.0).all())
