"""Host-only checks of how the 4-bit products are planned and of the limits of
their launches."""
import os

import pytest

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
