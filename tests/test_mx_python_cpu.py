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
