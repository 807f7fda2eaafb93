"""Every kind of output tile of the 4-bit products at sizes that really take it:
both tile heights, with more items than resident blocks, one step, two and many
along the contraction, whole tiles and edges, outputs into the caches and past
them, both types, plain, with dropout and added to what is there.

The fp32 product is compared with the float64 product of the values that the
operands stand for, all elements: K terms that are exact in fp32 are off by at
most K 2^-23 of the sum of their magnitudes, plus half a step of fp32.  The
other forms are functions of that fp32 product, rounded once, and have to equal
them bit for bit."""
import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from tests.gpu_helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mo._lib.load()


def _rand(rows, cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (x * torch.exp(torch.randn(rows, cols, generator=g, device="cuda"))).to(dtype)


def _close(got, qa, qb):
    """All elements of an fp32 product against float64, in strips of rows."""
    K = qa.cols
    a, b = mo.mx_dequantize(qa, dtype=F32).double(), mo.mx_dequantize(qb, dtype=F32).double().t().contiguous()
    size_b = b.abs()
    for r in range(0, qa.rows, 1024):
        exact, size = a[r:r + 1024] @ b, a[r:r + 1024].abs() @ size_b
        tol = K * 2.0 ** -23 * size
        tol += 2.0 ** -24 * (exact.abs() + tol)
        assert bool(((got[r:r + 1024].double() - exact).abs() <= tol).all()), r


# M, N, K, tile height, past the caches as (bf16, fp32), columns beside the output
CASES = [
    (8192, 8192, 128, 256, (False, True), 0),       # one step an item, whole tiles
    (10240, 10240, 256, 256, (True, True), 0),      # two steps
    (8191, 10240, 200, 256, (True, True), 5),       # edges along M, rows at any address
    (9001, 7003, 130, 256, (False, True), 5),       # edges along both
    (7900, 5003, 700, 256, (False, True), 0),
    (16384, 2560, 1100, 256, (False, True), 3),     # many steps, whole tiles at any address
    (8200, 8200, 130, 128, (True, True), 0),
    (4224, 4096, 520, 128, (False, False), 0),
]


@pytest.mark.parametrize("M,N,K,tile,past,beside", CASES)
def test_products_of_every_tile(M, N, K, tile, past, beside):
    for dt, far in zip((BF16, F32), past):
        info = mo.mx_plan_info([(M, N, K)], dt)
        assert (info["tile_rows"], info["parts"], info["past_caches"]) == (tile, [1], far)
        assert info["xcd_items"][-1] > 256 * (2 if tile == 256 else 3)
    announce(f"products of {tile}-high tiles {M}x{N}x{K}")
    qa, qb = mo.mx_quantize(_rand(M, K, BF16, 1)), mo.mx_quantize(_rand(N, K, BF16, 2))

    def run(dt, fill=None, **kw):
        buf = torch.full((M + 1, N + beside), 7.0, device="cuda", dtype=dt)
        out = buf[:M, :N]
        if fill is not None:
            out.copy_(fill)
        mo.mx_matmul(qa, qb, out=out, **kw)
        assert bool((buf[M:] == 7.0).all()) and bool((buf[:, N:] == 7.0).all())
        return out
    plain = run(F32)
    _close(plain, qa, qb)
    assert torch.equal(run(BF16), plain.to(BF16))
    dropped = mo.dropout(plain.contiguous(), 0.3, 99)
    for dt in (F32, BF16):
        assert torch.equal(run(dt, dropout=0.3, dropout_seed=99), dropped.to(dt))
        base = _rand(M, N, dt, 3)
        assert torch.equal(run(dt, base, accumulate=True), (base.float() + plain).to(dt))
        assert torch.equal(run(dt, base, accumulate=True, dropout=0.3, dropout_seed=99), (base.float() + dropped).to(dt))


def test_list_of_tall_tiles_with_empty_members():
    shapes = [(4000, 2048, 256)] * 3 + [(0, 2048, 256), (300, 2048, 0)] + [(4000, 2048, 256)] * 2
    info = mo.mx_plan_info(shapes)
    assert info["tile_rows"] == 256 and info["parts"] == [1, 1, 1, 0, 1, 1, 1]
    announce("list of tall tiles")
    qa = [mo.mx_quantize(_rand(m, k, BF16, 10 + i)) for i, (m, n, k) in enumerate(shapes)]
    qb = [mo.mx_quantize(_rand(n, k, BF16, 30 + i)) for i, (m, n, k) in enumerate(shapes)]
    plain = mo.mx_matmul(qa, qb, dtype=F32)
    for p, a, b in zip(plain, qa, qb):
        _close(p, a, b)
    assert all(torch.equal(p, q.to(BF16)) for p, q in zip(mo.mx_matmul(qa, qb), plain))
    # each member has the mask of its place in the list
    ones = [mo.mx_quantize(torch.ones(m, 32, device="cuda")) for m, n, k in shapes]
    wide = mo.mx_quantize(torch.ones(2048, 32, device="cuda"))
    keep = [m != 0 for m in mo.mx_matmul(ones, [wide] * len(shapes), dtype=F32, dropout=0.3, dropout_seed=5)]
    got = mo.mx_matmul(qa, qb, dtype=F32, dropout=0.3, dropout_seed=5)
    scale = (torch.tensor(65536.0) / (65536 - int(0.3 * 65536 + 0.5))).cuda()
    for g, p, k in zip(got, plain, keep):
        assert torch.equal(g, torch.where(k, p * scale, 0.0))
