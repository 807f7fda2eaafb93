"""Host-only checks of how the 4-bit products are planned and of the limits of
their launches."""
import os

import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import _lib

BASE = 0x7f0000000000   # fake device addresses: validation fails before any use
BF16, F32 = _lib.MUON_BF16, _lib.MUON_F32
E = _lib.CODES


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from orthogonalising_matrix_optimizer_amd import build
        build.build()
    return _lib.load()


def _arr(items):
    return (type(items[0]) * len(items))(*items)


def _operands(shapes):
    """Descriptors of the operands of M x N x K products, without memory."""
    return (_arr([_lib.MuonMX(None, None, m, k) for m, n, k in shapes]),
            _arr([_lib.MuonMX(None, None, n, k) for m, n, k in shapes]), len(shapes))


def test_split_lists_stay_inside_the_grids(lib):
    """The sum of a split product's parts takes a block for every 2048 elements
    and a launch at most 2^24 - 1 blocks: a list with a larger product is not
    split, however long another one's contraction is."""
    long = (128, 128, 1 << 24)
    assert lib.muon_mx_matmul_workspace_bytes(*_operands([long])) > 0
    for m, n in ((1 << 18, 1 << 17), ((1 << 18) + 5, (1 << 17) - 1)):
        assert m * (-(-n // 8)) > ((1 << 24) - 1) * 256
        assert lib.muon_mx_matmul_workspace_bytes(*_operands([(m, n, 128), long])) == 0
    below = (1 << 17, 1 << 17, 128)
    assert lib.muon_mx_matmul_workspace_bytes(*_operands([below, long])) > 0


def test_the_product_of_few_rows_refuses_what_its_grid_cannot_hold(lib):
    """512 threads for every 64 rows of b, below 2^32 threads a launch."""
    for rows in ((1 << 29) - 63, 1 << 29, 1 << 30):
        assert -(-rows // 64) * 512 >= 1 << 32
        x = _lib.MuonMat(BASE, 1, 96, 96, BF16, 0)
        b = _lib.MuonMX(BASE + (1 << 20), BASE + (1 << 40), rows, 96)
        out = _lib.MuonMat(BASE + (1 << 42), 1, rows, rows, BF16, 0)
        assert lib.muon_mx_matmul_rows(_arr([x]), _arr([b]), _arr([out]), None) == E["MUON_E_SHAPE"]


def test_limits_match_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "muon.h")).read()
    assert f"#define MUON_MX_FEW_ROWS_MAX_N {_lib.MX_FEW_ROWS_MAX_N}\n" in text


def test_plan_info(lib):
    """The tile heights, parts and ranges that the measurements chose; the tests of
    each kind of tile rely on these."""
    assert mo.mx_plan_info([(16384, 10240, 2560)]) == dict(
        tile_rows=256, parts=[1], past_caches=True, xcd_items=[640 * i for i in range(9)])
    info = mo.mx_plan_info([(2048, 2560, 2560)], torch.float32)
    assert (info["tile_rows"], info["parts"], info["past_caches"]) == (128, [1], False)
    info = mo.mx_plan_info([(768, 768, 8192), (0, 768, 8192), (768, 768, 0)], torch.float32)
    assert info["tile_rows"] == 128 and info["parts"][0] > 1 and info["parts"][1:] == [0, 1]
    # a list of more than one launch: the ranges are the first one's
    info = mo.mx_plan_info([(256, 128, 128)] * 80)
    assert info["parts"] == [1] * 80 and info["xcd_items"][-1] == 36 * (256 // info["tile_rows"])
    assert mo.mx_plan_info([(0, 5, 7)])["xcd_items"] == [0] * 9


def test_plan_info_refusals(lib):
    def call(m=64, n=32, k=96, out=None, dt=F32, count=1):
        a, b, _ = _operands([(m, n, k)])
        o = _arr([_lib.MuonMat(None, *(out or (m, n)), n, dt, 0)])
        return lib.muon_mx_plan_info(a, b, o, count, None, None, None, None)
    assert call() == 0
    assert call(count=0) == E["MUON_E_SHAPE"] and call(m=-1) == E["MUON_E_SHAPE"]
    assert call(out=(64, 33)) == E["MUON_E_SHAPE"] and call(k=(1 << 24) + 1) == E["MUON_E_SHAPE"]
    assert call(dt=9) == E["MUON_E_DTYPE"]
    a, b, _ = _operands([(1, 1, 1)])
    assert lib.muon_mx_plan_info(a, b, None, 1, None, None, None, None) == E["MUON_E_NULL"]
    with pytest.raises(_lib.MuonError):
        mo.mx_plan_info([])
    with pytest.raises(_lib.MuonError):
        mo.mx_plan_info([(-1, 5, 7)])


def _stages_by_xcd(shapes, info):
    """Steps of 128 columns that each XCD's items have, an empty item counting as one."""
    items = []
    for (m, n, k), parts in zip(shapes, info["parts"]):
        tiles, kt = -(-m // info["tile_rows"]) * -(-n // 128), -(-k // 128)
        chunk = -(-kt // parts) if parts else 0
        for p in range(parts):
            items += [max(1, min(chunk, kt - p * chunk))] * tiles
    edges = info["xcd_items"]
    assert edges[0] == 0 and edges[-1] == len(items) and edges == sorted(edges)
    return [sum(items[a:b]) for a, b in zip(edges, edges[1:])]


@pytest.mark.parametrize("shapes", [
    [(2048, 1408, 256 * (i % 2)) for i in range(36)],               # every second expert without tokens
    [(2048, 1408, 0)] * 5,                                          # none with any
    [(2048, 1408, 0)] * 18 + [(2048, 1408, 256)] * 18,
    [(2048, 1408, 256)] * 18 + [(2048, 1408, 0)] * 18,
    [(768, 768, 2000 * i) for i in range(12)],                      # split, the first one empty
    [(768, 768, 200 * (i % 3)) for i in range(30)] + [(768, 768, 30000)],
    [(1000 + 100 * i, 1408, 2048) for i in range(36)],
    [(16384, 10240, 2560)],
])
def test_work_is_dealt_evenly_to_the_xcds(lib, shapes):
    """An eighth of the steps each, within the longest item at either end.  A split
    product's items count with their mean length, and its last part is shorter:
    up to there its tiles have done as many steps more as that part lacks."""
    info = mo.mx_plan_info(shapes, torch.float32)
    stages = _stages_by_xcd(shapes, info)
    longest = short = 0
    for (m, n, k), parts in zip(shapes, info["parts"]):
        kt = -(-k // 128)
        chunk = -(-kt // max(1, parts))
        longest = max(longest, chunk, 1)
        if kt:
            short = max(short, -(-m // info["tile_rows"]) * -(-n // 128) * (chunk * parts - kt))
    assert max(abs(s - sum(stages) / 8) for s in stages) <= 2 * longest + short, (stages, info)
