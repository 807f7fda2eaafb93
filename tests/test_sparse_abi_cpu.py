"""Host-only checks of the embedding table's and the expert layers' C entries: struct
layouts, workspace sizes and the refusal of bad arguments before anything is enqueued."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import orthogonalising_matrix_optimizer_amd as mo
from orthogonalising_matrix_optimizer_amd import _lib, experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7f0000000000   # fake device addresses: validation fails before any use
BF16, F32 = _lib.MUON_BF16, _lib.MUON_F32
E = _lib.CODES
OK = 0


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

    def mat(self, r, c, dt=BF16, ld=None, ptr=None):
        ld = c if ld is None else ld
        return _lib.MuonMat(self.take(max(1, r * ld * 4)) if ptr is None else ptr, r, c, ld, dt, 0)

    def stack(self, n, r, c, dt=BF16, ld=None, stride=None, ptr=None):
        ld = c if ld is None else ld
        stride = r * ld if stride is None else stride
        return _lib.MuonStack(self.take(max(1, n * stride * 4)) if ptr is None else ptr, n, r, c, ld, stride, dt, 0)

    def slots(self, n=10, k=2, experts=4, **kw):
        s = _lib.MuonSlots(self.take(4 * experts + 4), self.take(4 * n * k), self.take(4 * n * k), n, k, experts)
        for f, v in kw.items():
            setattr(s, f, v)
        return s

    def ids(self, n, nbytes=8, ptr=None):
        return _lib.MuonIds(self.take(8 * n + 8) if ptr is None else ptr, n, nbytes, 0)


def ref(v):
    return None if v is None else ctypes.byref(v)


def test_struct_layout_matches_c_compiler():
    prog = r"""
#include <stdio.h>
#include <stddef.h>
#include "muon.h"
#define O(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
int main(void) {
  printf("muon_slots %zu\nmuon_stack %zu\nmuon_ids %zu\n", sizeof(muon_slots), sizeof(muon_stack), sizeof(muon_ids));
  O(muon_slots, offsets); O(muon_slots, tokens); O(muon_slots, place); O(muon_slots, n_tokens); O(muon_slots, k);
  O(muon_slots, experts);
  O(muon_stack, ptr); O(muon_stack, count); O(muon_stack, rows); O(muon_stack, cols); O(muon_stack, ld);
  O(muon_stack, stride); O(muon_stack, dtype);
  O(muon_ids, ptr); O(muon_ids, n); O(muon_ids, bytes);
  printf("limits %d,%d,%d\n", MUON_MAX_EXPERTS, MUON_MAX_K, MUON_MAX_SLOTS);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write(prog)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = dict(l.split() for l in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    assert got.pop("limits") == f"{_lib.MAX_EXPERTS},{_lib.MAX_K},{_lib.MAX_SLOTS}"
    ct = {"muon_slots": _lib.MuonSlots, "muon_stack": _lib.MuonStack, "muon_ids": _lib.MuonIds}
    for k, v in got.items():
        if "." in k:
            s, f = k.split(".")
            assert getattr(ct[s], f).offset == int(v), k
        else:
            assert ctypes.sizeof(ct[k]) == int(v), k
    # the packed descriptors of the Python layer are these structs
    assert (experts._SLOTS.size, experts._STACK.size, experts._IDS.size) == tuple(int(got[n]) for n in ct)


def test_workspace_sizes(lib):
    plan = lib.muon_expert_plan_workspace_bytes
    assert plan(0, 1, 4) == plan(1, 6, 64) == plan(500, 4, 64) == 0
    assert plan(16384, 6, 64) == 96 * 256 * 4                 # blocks of 1024 slots, 256 digits
    assert plan(16384, 6, 256) == 96 * 1024 * 4               # 257 keys: ten bits
    for bad in ((-1, 2, 4), (5, 0, 4), (5, 65, 4), (5, 2, 0), (5, 2, 513), (1 << 24, 2, 4)):
        assert plan(*bad) == 0
    grad = lib.muon_embedding_grad_workspace_bytes
    assert grad(0, 10, 10) == grad(256, 50257, 768) == 0      # a few tokens need none
    n = grad(16384, 50257, 768)                               # two keys and two places a token, counts, partial rows
    assert n == 4 * 65536 + 16 * 256 * 4 + 1024 * 2 * 768 * 4   # chunks of 16 tokens
    assert grad(300, 40, 33) == 4 * 1200 + 38 * 2 * 40 * 4    # rows of whole groups of eight
    for bad in ((-1, 5, 5), ((1 << 24) + 1, 5, 5), (5, -1, 5), (5, 1 << 30, 5), (5, 5, -1), (5, 5, (1 << 24) + 1)):
        assert grad(*bad) == 0


def test_plan_and_route_refusals(lib):
    room = Room()
    ids, slots = room.ids(20), room.slots()

    def plan(i=ids, s=slots, ws=None, size=0):
        return lib.muon_expert_plan(ref(i), ref(s), ws, size, None)
    assert plan(i=None) == E["MUON_E_NULL"] and plan(s=None) == E["MUON_E_NULL"]
    assert plan(i=room.ids(19)) == E["MUON_E_SHAPE"] and plan(i=room.ids(20, 2)) == E["MUON_E_DTYPE"]
    assert plan(i=room.ids(20, 8, ptr=BASE + 4)) == E["MUON_E_ALIGN"]
    assert plan(i=_lib.MuonIds(None, 20, 8, 0)) == E["MUON_E_NULL"]
    for kw in (dict(k=0), dict(k=65), dict(experts=0), dict(experts=513), dict(n_tokens=-1), dict(n_tokens=1 << 24)):
        assert plan(s=room.slots(**kw)) == E["MUON_E_SHAPE"], kw
    for f in ("offsets", "tokens", "place"):
        assert plan(s=room.slots(**{f: None})) == E["MUON_E_NULL"]
        assert plan(s=room.slots(**{f: BASE + 2})) == E["MUON_E_ALIGN"]
        assert plan(s=room.slots(**{f: ids.ptr})) == E["MUON_E_ALIAS"]
    assert plan(s=room.slots(tokens=slots.tokens, place=slots.tokens + 76)) == E["MUON_E_ALIAS"]
    big, many = room.slots(20000, 2, 4), room.ids(40000)
    need = lib.muon_expert_plan_workspace_bytes(20000, 2, 4)
    assert need and plan(many, big) == E["MUON_E_WORKSPACE"]
    assert plan(many, big, room.take(need), need - 1) == E["MUON_E_WORKSPACE"]
    assert plan(many, big, room.take(need) + 8, need) == E["MUON_E_ALIGN"]
    assert plan(many, big, many.ptr, need) == E["MUON_E_ALIAS"]

    x, gates, chosen = room.mat(10, 4, F32), room.take(80), room.take(80)

    def route(l=x, g=gates, c=chosen, s=slots):
        return lib.muon_route(ref(l), 0, g, c, ref(s), None, 0, None)
    assert route(l=None) == E["MUON_E_NULL"] and route(g=None) == E["MUON_E_NULL"] and route(c=None) == E["MUON_E_NULL"]
    assert route(l=room.mat(9, 4)) == E["MUON_E_SHAPE"] and route(l=room.mat(10, 5)) == E["MUON_E_SHAPE"]
    assert route(l=room.mat(10, 4, 5)) == E["MUON_E_DTYPE"] and route(l=room.mat(10, 4, ld=3)) == E["MUON_E_SHAPE"]
    assert route(g=gates + 2) == E["MUON_E_ALIGN"] and route(c=gates) == E["MUON_E_ALIAS"]
    assert route(g=x.ptr) == E["MUON_E_ALIAS"] and route(c=slots.place) == E["MUON_E_ALIAS"]

    dg, out = room.take(80), room.mat(10, 4, F32)

    def grad(d=dg, l=x, g=gates, c=chosen, k=2, o=out):
        return lib.muon_route_grad(d, ref(l), g, c, k, 0, ref(o), None)
    assert grad(d=None) == grad(l=None) == grad(g=None) == grad(c=None) == grad(o=None) == E["MUON_E_NULL"]
    assert grad(o=room.mat(10, 5)) == E["MUON_E_SHAPE"] and grad(k=0) == E["MUON_E_SHAPE"] and grad(k=65) == E["MUON_E_SHAPE"]
    assert grad(d=dg + 1) == E["MUON_E_ALIGN"] and grad(o=x) == E["MUON_E_ALIAS"]
    assert grad(l=room.mat(0, 4), o=room.mat(0, 4)) == OK


def test_product_refusals(lib):
    room = Room()
    slots, w = room.slots(), room.stack(4, 24, 40)
    x, xt, y = room.mat(20, 40), room.mat(10, 40), room.mat(20, 24)

    def fwd(x=x, w=w, s=slots, gather=0, o=y):
        return lib.muon_expert_linear(ref(x), ref(w), ref(s), gather, ref(o), None)
    assert fwd(x=None) == fwd(w=None) == fwd(s=None) == fwd(o=None) == E["MUON_E_NULL"]
    assert fwd(x=xt) == E["MUON_E_SHAPE"] and fwd(gather=1) == E["MUON_E_SHAPE"]      # tokens' rows and slots' rows
    assert fwd(x=room.mat(20, 41)) == E["MUON_E_SHAPE"] and fwd(o=room.mat(20, 23)) == E["MUON_E_SHAPE"]
    assert fwd(o=room.mat(19, 24)) == E["MUON_E_SHAPE"] and fwd(w=room.stack(5, 24, 40)) == E["MUON_E_SHAPE"]
    assert fwd(x=room.mat(20, 40, F32)) == E["MUON_E_DTYPE"] and fwd(w=room.stack(4, 24, 40, 3)) == E["MUON_E_DTYPE"]
    assert fwd(o=room.mat(20, 24, 3)) == E["MUON_E_DTYPE"]
    assert fwd(w=room.stack(4, 24, 40, ld=39)) == E["MUON_E_SHAPE"]
    assert fwd(w=room.stack(4, 24, 40, stride=24 * 40 - 1)) == E["MUON_E_SHAPE"]      # matrices that overlap
    assert fwd(w=room.stack(4, 24, 40, ptr=BASE + 1)) == E["MUON_E_ALIGN"]
    assert fwd(w=_lib.MuonStack(None, 4, 24, 40, 40, 960, BF16, 0)) == E["MUON_E_NULL"]
    assert fwd(o=room.mat(20, 24, ptr=x.ptr)) == E["MUON_E_ALIAS"]
    assert fwd(o=room.mat(20, 24, ptr=w.ptr + 4 * 24 * 40 * 2 - 2)) == E["MUON_E_ALIAS"]
    assert fwd(o=room.mat(20, 24, ptr=slots.offsets)) == E["MUON_E_ALIAS"]
    # a gathered x that is too long to be addressed, and the same not gathered
    far = room.slots(1 << 20, 1)
    wide, out = room.stack(4, 8, 2048), room.mat(1 << 20, 8)
    long = room.mat(1 << 20, 2048)
    assert fwd(long, wide, far, 1, out) == E["MUON_E_SHAPE"]
    none = room.slots(0)
    assert fwd(room.mat(0, 40), w, none, 0, room.mat(0, 24)) == OK

    dx = room.mat(20, 40)

    def back(d=y, w=w, s=slots, o=dx):
        return lib.muon_expert_linear_dx(ref(d), ref(w), ref(s), ref(o), None)
    assert back(d=None) == back(w=None) == back(s=None) == back(o=None) == E["MUON_E_NULL"]
    assert back(d=x) == E["MUON_E_SHAPE"] and back(o=y) == E["MUON_E_SHAPE"]
    assert back(o=room.mat(20, 40, ptr=y.ptr)) == E["MUON_E_ALIAS"]

    dw = room.stack(4, 24, 40, F32)

    def weights(d=y, x=x, s=slots, gather=0, o=dw):
        return lib.muon_expert_linear_dw(ref(d), ref(x), ref(s), gather, 0, ref(o), None, 0, None)
    assert weights(d=None) == weights(x=None) == weights(s=None) == weights(o=None) == E["MUON_E_NULL"]
    assert weights(x=xt) == E["MUON_E_SHAPE"] and weights(gather=1) == E["MUON_E_SHAPE"]
    assert weights(o=room.stack(4, 40, 24, F32)) == E["MUON_E_SHAPE"] and weights(o=room.stack(3, 24, 40)) == E["MUON_E_SHAPE"]
    assert weights(d=room.mat(20, 24, F32)) == E["MUON_E_DTYPE"]
    assert weights(o=room.stack(4, 24, 40, F32, ptr=x.ptr)) == E["MUON_E_ALIAS"]


def test_combine_refusals(lib):
    room = Room()
    slots, y, out, gates = room.slots(), room.mat(20, 40), room.mat(10, 40), room.take(80)

    def fwd(y=y, g=gates, s=slots, o=out):
        return lib.muon_expert_combine(ref(y), g, ref(s), ref(o), None)
    assert fwd(y=None) == fwd(s=None) == fwd(o=None) == E["MUON_E_NULL"]
    assert fwd(y=out) == E["MUON_E_SHAPE"] and fwd(o=y) == E["MUON_E_SHAPE"] and fwd(o=room.mat(10, 41)) == E["MUON_E_SHAPE"]
    assert fwd(g=gates + 2) == E["MUON_E_ALIGN"] and fwd(o=room.mat(10, 40, ptr=y.ptr)) == E["MUON_E_ALIAS"]
    assert fwd(g=out.ptr) == E["MUON_E_ALIAS"] and fwd(o=room.mat(10, 40, 9)) == E["MUON_E_DTYPE"]

    dy, dg = room.mat(20, 40), room.take(80)

    def back(d=out, y=y, g=gates, s=slots, o=dy, dg=dg):
        return lib.muon_expert_combine_grad(ref(d), ref(y), g, ref(s), ref(o), dg, None)
    assert back(d=None) == back(y=None) == back(s=None) == E["MUON_E_NULL"]
    assert back(d=y) == E["MUON_E_SHAPE"] and back(o=out) == E["MUON_E_SHAPE"] and back(y=room.mat(20, 39)) == E["MUON_E_SHAPE"]
    assert back(y=room.mat(20, 40, F32)) == E["MUON_E_DTYPE"] and back(o=room.mat(20, 40, F32)) == E["MUON_E_DTYPE"]
    assert back(o=y) == E["MUON_E_ALIAS"] and back(dg=gates) == E["MUON_E_ALIAS"] and back(dg=dg + 1) == E["MUON_E_ALIGN"]
    assert back(o=None, dg=None) == OK
    assert lib.muon_expert_gather(ref(out), ref(slots), None, None) == E["MUON_E_NULL"]
    assert lib.muon_expert_gather(ref(y), ref(slots), ref(dy), None) == E["MUON_E_SHAPE"]


def test_embedding_refusals(lib):
    room = Room()
    ids, w, out = room.ids(20), room.mat(100, 40), room.mat(20, 40)

    def fwd(i=ids, w=w, s=1.0, o=out):
        return lib.muon_embedding(ref(i), ref(w), s, ref(o), None)
    assert fwd(i=None) == fwd(w=None) == fwd(o=None) == E["MUON_E_NULL"]
    assert fwd(o=room.mat(19, 40)) == E["MUON_E_SHAPE"] and fwd(o=room.mat(20, 39)) == E["MUON_E_SHAPE"]
    assert fwd(o=room.mat(20, 40, F32)) == E["MUON_E_DTYPE"] and fwd(i=room.ids(20, 1)) == E["MUON_E_DTYPE"]
    assert fwd(i=room.ids((1 << 24) + 1)) == E["MUON_E_SHAPE"]
    for s in (float("nan"), float("inf")):
        assert fwd(s=s) == E["MUON_E_HPARAM"]
    assert fwd(o=room.mat(20, 40, ptr=w.ptr)) == E["MUON_E_ALIAS"] and fwd(o=room.mat(20, 40, ptr=ids.ptr)) == E["MUON_E_ALIAS"]
    assert fwd(i=room.ids(0), o=room.mat(0, 40)) == OK

    dy, dw = room.mat(20, 40), room.mat(100, 40, F32)

    def back(d=dy, i=ids, s=1.0, o=dw, ws=None, size=0):
        return lib.muon_embedding_grad(ref(d), ref(i), s, 0, ref(o), ws, size, None)
    assert back(d=None) == back(i=None) == back(o=None) == E["MUON_E_NULL"]
    assert back(d=room.mat(19, 40)) == E["MUON_E_SHAPE"] and back(o=room.mat(100, 41, F32)) == E["MUON_E_SHAPE"]
    assert back(s=float("nan")) == E["MUON_E_HPARAM"] and back(o=room.mat(100, 40, F32, ptr=dy.ptr)) == E["MUON_E_ALIAS"]
    d, i = room.mat(300, 40), room.ids(300)
    need = lib.muon_embedding_grad_workspace_bytes(300, 100, 40)
    assert back(d, i) == E["MUON_E_WORKSPACE"] and back(d, i, ws=room.take(need), size=need - 1) == E["MUON_E_WORKSPACE"]
    assert back(d, i, ws=dw.ptr, size=need) == E["MUON_E_ALIAS"] and back(d, i, ws=BASE + 8, size=need) == E["MUON_E_ALIGN"]


def test_memory_of_split_contractions(lib):
    """Few tiles and many rows need memory, which is checked; the rest needs none."""
    room = Room()

    def need(slots, dw):
        return lib.muon_expert_linear_dw_workspace_bytes(slots, ref(dw))
    dw = room.stack(2, 100, 61, F32)
    assert need(200, dw) == need(0, dw) == 0
    n = need(8000, dw)
    assert n > 0 and n % (100 * 64 * 4) == 0
    assert need(8000, room.stack(64, 100, 61, F32)) == need(8000, room.stack(2, 2048, 2048, F32)) == 0
    assert need(8000, room.stack(2, 0, 61, F32)) == need(-1, dw) == need(1 << 40, dw) == need(8000, None) == 0
    assert 0 < need(_lib.MAX_SLOTS, room.stack(1, 64, 64, F32)) < 1 << 28
    slots = room.slots(4000, 2, 2)
    d, x = room.mat(8000, 100), room.mat(8000, 61)

    def call(ws, size, o=dw):
        return lib.muon_expert_linear_dw(ref(d), ref(x), ref(slots), 0, 0, ref(o), ws, size, None)
    assert call(None, 0) == call(room.take(n), n - 1) == E["MUON_E_WORKSPACE"]
    assert call(BASE + 8, n) == E["MUON_E_ALIGN"]
    assert call(dw.ptr, n) == call(x.ptr, n) == E["MUON_E_ALIAS"]


def test_package_exports():
    for n in ("route", "route_grad", "expert_plan", "expert_gather", "expert_linear", "expert_linear_grad", "expert_combine",
              "expert_combine_grad", "embedding", "embedding_grad", "ExpertPlan", "Routing"):
        assert n in mo.__all__ and hasattr(mo, n)
