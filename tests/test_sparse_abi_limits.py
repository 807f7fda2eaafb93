"""Descriptors of the embedding's and the expert layers' C entries at and past their limits,
host-only: sizes whose products pass 64 bits are refused, not taken for small ones."""
import pytest

from orthogonalising_matrix_optimizer_amd import _lib
from tests.test_sparse_abi_cpu import BF16, E, F32, Room, lib, ref  # noqa: F401 (lib is a fixture)

ROWS, PITCH = 1 << 24, 1 << 40      # the most rows of these operators' matrices, the largest pitch of any


def test_gradients_of_matrices_past_the_address_space(lib):
    """dw of which rows times pitch passes 64 bits, with strides that the wrapped product allows."""
    room = Room()
    slots, dy, x = room.slots(n=10, k=2, experts=2), room.mat(20, ROWS, ld=ROWS, ptr=1 << 45), room.mat(20, 8)

    def dw(ld, stride, rows=ROWS, count=2):
        d = dy if rows == ROWS else room.mat(20, rows)
        w = _lib.MuonStack(1 << 44, count, rows, 8, ld, stride, F32, 0)
        s = slots if count == 2 else room.slots(n=10, k=2, experts=count)
        return lib.muon_expert_linear_dw(ref(d), ref(x), ref(s), 0, 0, ref(w), None, 0, None)
    for stride in (0, 1 << 49, (ROWS - 1) * PITCH + 8 - (1 << 64), -1):
        assert dw(PITCH, stride) == E["MUON_E_SHAPE"], stride
    assert dw(PITCH, 0, count=1) == E["MUON_E_SHAPE"]
    assert dw(PITCH + 1, 1 << 50, rows=2) == E["MUON_E_SHAPE"]
    assert dw(8, (1 << 63) - 1, rows=2) == E["MUON_E_SHAPE"] and dw(8, 1 << 56, rows=2) == E["MUON_E_SHAPE"]


def test_rows_past_the_address_space(lib):
    """Matrices whose last row's offset wraps: nothing could be said of what they share memory with."""
    room = Room()
    slots, w, x = room.slots(n=ROWS, k=1, experts=4), room.stack(4, 8, 8), room.mat(ROWS, 8)
    far = room.mat(ROWS, 8, ld=PITCH, ptr=1 << 44)
    assert lib.muon_expert_linear(ref(x), ref(w), ref(slots), 0, ref(far), None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_linear(ref(far), ref(w), ref(slots), 1, ref(x), None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_linear_dx(ref(far), ref(w), ref(slots), ref(x), None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_combine(ref(x), None, ref(slots), ref(far), None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_combine(ref(far), None, ref(slots), ref(x), None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_gather(ref(far), ref(slots), ref(x), None) == E["MUON_E_SHAPE"]
    ids = room.ids(20)
    table, out = room.mat(1 << 30, 8, ld=PITCH, ptr=1 << 44), room.mat(20, 8)
    assert lib.muon_embedding(ref(ids), ref(table), 1.0, ref(out), None) == E["MUON_E_SHAPE"]
    assert lib.muon_embedding_grad(ref(out), ref(ids), 1.0, 0, ref(table), None, 0, None) == E["MUON_E_SHAPE"]
    logits = room.mat(ROWS, 4, F32, ld=PITCH, ptr=1 << 44)
    gates, chosen = 1 << 42, 1 << 43
    assert lib.muon_route(ref(logits), 0, gates, chosen, ref(slots), None, 0, None) == E["MUON_E_SHAPE"]
    small = room.mat(ROWS, 4, F32)
    assert lib.muon_route_grad(gates, ref(logits), 1 << 41, chosen, 1, 0, ref(small), None) == E["MUON_E_SHAPE"]


@pytest.mark.parametrize("tokens", [(1 << 24) + 1, 1 << 58, 1 << 62, (1 << 63) - 1, -(1 << 63)])
def test_numbers_of_tokens_past_64_bits(lib, tokens):
    room = Room()
    slots = _lib.MuonSlots(room.take(64), room.take(64), room.take(64), tokens, 64, 4)
    assert lib.muon_expert_plan(ref(room.ids(20)), ref(slots), None, 0, None) == E["MUON_E_SHAPE"]
    assert lib.muon_expert_plan_workspace_bytes(tokens, 64, 4) == 0
    assert lib.muon_expert_linear(ref(room.mat(20, 8)), ref(room.stack(4, 8, 8)), ref(slots), 0, ref(room.mat(20, 8)),
                                  None) == E["MUON_E_SHAPE"]


def test_largest_descriptors_are_still_compared(lib):
    """Just inside the limits an overlap is seen."""
    room = Room()
    slots, dy, x = room.slots(n=10, k=2, experts=2), room.mat(20, 1 << 11), room.mat(20, 8)
    base = 1 << 50
    stride = (1 << 11) * PITCH // 2
    last = base + 4 * (stride + ((1 << 11) - 1) * (PITCH // 2))

    def dw(o):
        return lib.muon_expert_linear_dw(ref(dy), ref(o), ref(slots), 0, 0,
                                         ref(_lib.MuonStack(base, 2, 1 << 11, 8, PITCH // 2, stride, F32, 0)), None, 0, None)
    assert dw(room.mat(20, 8, ptr=last)) == E["MUON_E_ALIAS"]
    assert dw(room.mat(20, 8, BF16, ptr=base)) == E["MUON_E_ALIAS"]
