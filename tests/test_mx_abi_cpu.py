"""Host-only checks of the 4-bit operators and dropout: storage sizes, struct
layouts, and the refusal of bad arguments before anything is enqueued."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7f0000000000   # fake device addresses: validation fails before any use
BF16, F32 = _lib.MUON_BF16, _lib.MUON_F32
E = _lib.CODES


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from orthogonalising_matrix_optimizer_amd import build
        build.build()
    return _lib.load()


class Room:
    """Hands out fake device addresses that do not overlap."""

    def __init__(self):
        self.at = BASE

    def take(self, nbytes):
        a = self.at
        self.at += (nbytes + 4095) // 4096 * 4096 + 4096
        return a


def _mat(room, r, c, dt=BF16, ld=None, ptr=None):
    ld = c if ld is None else ld
    if ptr is None:
        ptr = room.take(max(1, r * ld * 4))
    return _lib.MuonMat(ptr, r, c, ld, dt, 0)


def _mx(lib, room, r, c):
    return _lib.MuonMX(room.take(lib.muon_mx_codes_bytes(r, c) + 1), room.take(lib.muon_mx_scales_bytes(r, c) + 1), r, c)


def _arr(items):
    return (type(items[0]) * len(items))(*items)


def test_struct_layout_matches_c_compiler():
    prog = r"""
#include <stdio.h>
#include <stddef.h>
#include "muon.h"
#define O(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
int main(void) {
  printf("muon_mx %zu\nmuon_mx_options %zu\nmuon_mat %zu\n", sizeof(muon_mx), sizeof(muon_mx_options), sizeof(muon_mat));
  O(muon_mx, codes); O(muon_mx, scales); O(muon_mx, rows); O(muon_mx, cols);
  O(muon_mx_options, stochastic); O(muon_mx_options, accumulate); O(muon_mx_options, dropout);
  O(muon_mx_options, seed); O(muon_mx_options, dropout_seed); O(muon_mx_options, seed_dev);
  O(muon_mx_options, dropout_seed_dev);
  printf("few %d\n", MUON_MX_FEW_ROWS);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write(prog)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = dict(l.split() for l in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got.pop("few")) == _lib.MX_FEW_ROWS
    ct = {"muon_mx": _lib.MuonMX, "muon_mx_options": _lib.MXOptions, "muon_mat": _lib.MuonMat}
    for k, v in got.items():
        if "." in k:
            s, f = k.split(".")
            assert getattr(ct[s], f).offset == int(v), k
        else:
            assert ctypes.sizeof(ct[k]) == int(v), k
    # the packed descriptors of the Python layer are these structs
    assert mo.mx._MAT1.size == ctypes.sizeof(_lib.MuonMat) and mo.mx._MX1.size == ctypes.sizeof(_lib.MuonMX)


@pytest.mark.parametrize("r,c", [(0, 0), (0, 5), (5, 0), (1, 1), (16, 128), (17, 129), (64, 4096), (65, 4097), (1000, 333)])
def test_storage_bytes(lib, r, c):
    codes, scales = lib.muon_mx_codes_bytes(r, c), lib.muon_mx_scales_bytes(r, c)
    assert codes == -(-r // 16) * -(-c // 128) * 1024
    assert scales == -(-r // 64) * -(-c // 128) * 256
    assert mo.mx._mx_bytes(r, c) == codes + scales


def test_storage_bytes_of_impossible_shapes(lib):
    for r, c in ((-1, 5), (5, -1), ((1 << 30) + 1, 1), (1, (1 << 24) + 1)):
        assert lib.muon_mx_codes_bytes(r, c) == 0 and lib.muon_mx_scales_bytes(r, c) == 0


def test_quantize_refusals(lib):
    room = Room()
    x, q, t = _mat(room, 64, 96), _mx(lib, room, 64, 96), _mx(lib, room, 96, 64)

    def call(i=(x,), o=(q,), ot=(t,), n=1, opt=None):
        return lib.muon_mx_quantize(_arr(list(i)) if i else None, _arr(list(o)) if o else None,
                                    _arr(list(ot)) if ot else None, n, opt, None)
    assert call(n=-1) == E["MUON_E_SHAPE"]
    assert call(n=0) == 0
    assert call(i=None) == E["MUON_E_NULL"]
    assert call(o=None, ot=None) == E["MUON_E_NULL"]
    assert call(i=(_mat(room, 64, 96, dt=7),)) == E["MUON_E_DTYPE"]
    assert call(i=(_mat(room, 64, 96, ld=95),)) == E["MUON_E_SHAPE"]
    assert call(i=(_mat(room, 64, 96, ld=0),)) == E["MUON_E_SHAPE"]
    assert call(i=(_mat(room, 65, 96),)) == E["MUON_E_SHAPE"]
    assert call(i=(_mat(room, -1, 96),)) == E["MUON_E_SHAPE"]
    assert call(i=(_lib.MuonMat(None, 64, 96, 96, BF16, 0),)) == E["MUON_E_NULL"]
    assert call(i=(_lib.MuonMat(x.ptr + 1, 64, 96, 96, BF16, 0),)) == E["MUON_E_ALIGN"]
    assert call(o=(_lib.MuonMX(q.codes + 8, q.scales, 64, 96),)) == E["MUON_E_ALIGN"]
    assert call(o=(_lib.MuonMX(q.codes, None, 64, 96),)) == E["MUON_E_NULL"]
    assert call(ot=(_mx(lib, room, 64, 96),)) == E["MUON_E_SHAPE"]
    assert call(o=(_lib.MuonMX(x.ptr, q.scales, 64, 96),)) == E["MUON_E_ALIAS"]
    assert call(o=(q,), ot=(_lib.MuonMX(q.codes, t.scales, 96, 64),)) == E["MUON_E_ALIAS"]
    # the same output twice in a list, and two element types
    assert call(i=(x, x), o=(q, q), ot=None, n=2) == E["MUON_E_ALIAS"]
    assert call(i=(x, _mat(room, 64, 96, F32)), o=(q, _mx(lib, room, 64, 96)), ot=None, n=2) == E["MUON_E_DTYPE"]
    for p in (-0.1, 1.0, 0.999999, float("nan"), float("inf")):
        assert call(opt=_lib.MXOptions(dropout=p)) == E["MUON_E_HPARAM"]
    assert call(opt=_lib.MXOptions(stochastic=1, seed_dev=BASE + 4)) == E["MUON_E_ALIGN"]
    assert call(opt=_lib.MXOptions(stochastic=1, seed_dev=q.codes)) == E["MUON_E_ALIAS"]
    # beyond the grid
    big = _lib.MuonMat(BASE, 1 << 30, 1 << 24, 1 << 24, BF16, 0)
    assert call(i=(big,), o=(_lib.MuonMX(BASE, BASE, 1 << 30, 1 << 24),), ot=None) == E["MUON_E_SHAPE"]


def test_empty_matrices_need_no_memory(lib):
    e = _lib.MuonMat(None, 0, 96, 96, BF16, 0)
    q, t = _lib.MuonMX(None, None, 0, 96), _lib.MuonMX(None, None, 96, 0)
    assert lib.muon_mx_quantize(_arr([e]), _arr([q]), _arr([t]), 1, None, None) == 0
    assert lib.muon_mx_dequantize(_arr([q]), _arr([e]), 1, None) == 0
    w = _lib.MuonMX(None, None, 0, 96)
    assert lib.muon_mx_matmul(_arr([q]), _arr([w]), _arr([_lib.MuonMat(None, 0, 0, 0, F32, 0)]), 1, None, None, 0, None) == 0
    assert lib.muon_mx_matmul_rows(_arr([e]), _arr([w]), _arr([_lib.MuonMat(None, 0, 0, 0, F32, 0)]), None) == 0
    assert lib.muon_dropout(_arr([e]), _arr([e]), 0.5, 1, None, None) == 0


def test_matmul_refusals(lib):
    room = Room()
    a, b, o = _mx(lib, room, 64, 96), _mx(lib, room, 32, 96), _mat(room, 64, 32, F32)

    def call(x=(a,), y=(b,), z=(o,), n=1, opt=None, ws=None, wb=0):
        return lib.muon_mx_matmul(_arr(list(x)) if x else None, _arr(list(y)) if y else None,
                                  _arr(list(z)) if z else None, n, opt, ws, wb, None)
    assert call(n=-1) == E["MUON_E_SHAPE"]
    assert call(x=None) == E["MUON_E_NULL"] and call(z=None) == E["MUON_E_NULL"]
    assert call(y=(_mx(lib, room, 32, 97),)) == E["MUON_E_SHAPE"]
    assert call(z=(_mat(room, 64, 33, F32),)) == E["MUON_E_SHAPE"]
    assert call(z=(_mat(room, 64, 32, ld=31),)) == E["MUON_E_SHAPE"]
    assert call(z=(_mat(room, 64, 32, 9),)) == E["MUON_E_DTYPE"]
    assert call(z=(_lib.MuonMat(a.codes, 64, 32, 32, F32, 0),)) == E["MUON_E_ALIAS"]
    assert call(x=(a, a), y=(b, b), z=(o, o), n=2) == E["MUON_E_ALIAS"]
    assert call(x=(a, a), y=(b, b), z=(o, _mat(room, 64, 32)), n=2) == E["MUON_E_DTYPE"]
    assert call(opt=_lib.MXOptions(dropout=2.0)) == E["MUON_E_HPARAM"]
    # overlapping column slices of one buffer
    p = room.take(64 * 100 * 4)
    s1, s2 = _lib.MuonMat(p, 64, 32, 100, F32, 0), _lib.MuonMat(p + 31 * 4, 64, 32, 100, F32, 0)
    assert call(x=(a, a), y=(b, b), z=(s1, s2), n=2) == E["MUON_E_ALIAS"]
    # a split contraction wants its workspace
    la, lb, lo = _mx(lib, room, 128, 65536), _mx(lib, room, 128, 65536), _mat(room, 128, 128, F32)
    need = lib.muon_mx_matmul_workspace_bytes(_arr([la]), _arr([lb]), 1)
    assert need >= 2 * 128 * 128 * 4
    assert call(x=(la,), y=(lb,), z=(lo,)) == E["MUON_E_WORKSPACE"]
    ws = room.take(need)
    assert call(x=(la,), y=(lb,), z=(lo,), ws=ws, wb=need - 1) == E["MUON_E_WORKSPACE"]
    assert call(x=(la,), y=(lb,), z=(lo,), ws=ws + 8, wb=need) == E["MUON_E_ALIGN"]
    assert call(x=(la,), y=(lb,), z=(lo,), ws=lo.ptr, wb=need) == E["MUON_E_ALIAS"]
    # lists that are not split, and arguments without a plan
    assert lib.muon_mx_matmul_workspace_bytes(_arr([a]), _arr([b]), 1) == 0
    assert lib.muon_mx_matmul_workspace_bytes(None, None, 1) == 0
    assert lib.muon_mx_matmul_workspace_bytes(_arr([a]), _arr([_mx(lib, room, 3, 4)]), 1) == 0


def test_rows_and_dropout_refusals(lib):
    room = Room()
    x, w, o = _mat(room, 16, 96), _mx(lib, room, 32, 96), _mat(room, 16, 32)

    def rows(a=x, b=w, c=o):
        return lib.muon_mx_matmul_rows(_arr([a]) if a else None, _arr([b]), _arr([c]), None)
    assert rows(a=None) == E["MUON_E_NULL"]
    assert rows(a=_mat(room, 17, 96), c=_mat(room, 17, 32)) == E["MUON_E_SHAPE"]
    assert rows(a=_mat(room, 16, 95)) == E["MUON_E_SHAPE"]
    assert rows(c=_mat(room, 16, 33)) == E["MUON_E_SHAPE"]
    assert rows(c=_lib.MuonMat(x.ptr, 16, 32, 32, BF16, 0)) == E["MUON_E_ALIAS"]

    y = _mat(room, 16, 96)

    def drop(a=x, b=y, p=0.5, dev=None):
        return lib.muon_dropout(_arr([a]) if a else None, _arr([b]), p, 1, dev, None)
    assert drop(a=None) == E["MUON_E_NULL"]
    assert drop(b=_mat(room, 16, 96, F32)) == E["MUON_E_DTYPE"]
    assert drop(b=_mat(room, 16, 95)) == E["MUON_E_SHAPE"]
    assert drop(b=_lib.MuonMat(x.ptr + 32, 16, 96, 96, BF16, 0)) == E["MUON_E_ALIAS"]
    assert drop(dev=BASE + 4) == E["MUON_E_ALIGN"]
    for p in (-1.0, 1.0, float("nan")):
        assert drop(p=p) == E["MUON_E_HPARAM"]


def test_python_layer_refuses_before_the_library():
    cpu = torch.zeros(4, 8)
    for f in (lambda: mo.mx_quantize(cpu), lambda: mo.dropout(cpu, 0.1, 1), lambda: mo.mx_quantize([cpu, 3]),
              lambda: mo.mx_quantize(cpu, "sideways"), lambda: mo.mx_quantize(torch.tensor(1.0))):
        with pytest.raises(ValueError):
            f()
    assert mo.mx_quantize([]) == [] and mo.mx_dequantize([]) == [] and mo.mx_matmul([], []) == []
