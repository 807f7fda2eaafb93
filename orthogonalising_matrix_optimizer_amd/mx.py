"""4-bit operators and dropout: torch-facing wrappers of the C ABI.

Quantisation to microscaled 4-bit blocks, reading back, products over lists of
matrices, the linear layer with its gradients, and dropout whose mask is a
function of a seed and is never stored.  The number format and the random
numbers are stated in include/muon.h.  As in the rest of the package all
computation runs in the HIP library; this module allocates outputs and passes
pointers with the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import List, NamedTuple, Optional, Sequence, Tuple, Union

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.MUON_BF16, torch.float32: _lib.MUON_F32}

Seed = Union[int, torch.Tensor]


class MX4:
    """A rows x cols matrix in 4 bits (blocks of 32 along the columns share a scale).

    `data` holds codes and scales in the order in which the matrix
    instructions read them; use mx_dequantize for values."""

    __slots__ = ("data", "rows", "cols", "c")

    def __init__(self, rows: int, cols: int, device):
        lib = _lib.load()
        codes = int(lib.muon_mx_codes_bytes(rows, cols))
        if codes == 0 and rows * cols != 0:
            raise ValueError(f"no 4-bit matrix of shape {rows} x {cols}")
        self.data = torch.empty(codes + int(lib.muon_mx_scales_bytes(rows, cols)), dtype=torch.uint8,
                                device=device)
        self.rows, self.cols = rows, cols
        p = self.data.data_ptr()
        self.c = _lib.MuonMX(p if codes else None, p + codes if codes else None, rows, cols)

    @property
    def shape(self) -> Tuple[int, int]:
        return (self.rows, self.cols)

    @property
    def device(self) -> torch.device:
        return self.data.device

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return mx_dequantize(self, dtype)

    def __repr__(self) -> str:
        return f"MX4({self.rows} x {self.cols}, {self.device})"


class MXPair(NamedTuple):
    """A matrix in 4 bits and its transpose in 4 bits."""
    w: MX4
    w_t: MX4


class MXSaved(NamedTuple):
    """What mx_linear keeps for mx_linear_grad: the input's transpose in 4 bits
    (after dropout) and how to make the dropout mask again."""
    x_t: MX4
    dropout: float
    dropout_seed: Optional[Seed]


def _rows_of(t: torch.Tensor) -> torch.Tensor:
    """`t` as a 2-D view of its rows (last dimension)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"expected a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU")
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError("tensors must have at least one dimension")
    try:
        return t.view(t.numel() // t.shape[-1] if t.shape[-1] else 0, t.shape[-1])
    except RuntimeError:
        raise ValueError("the leading dimensions must be one run of evenly spaced rows") from None


def _mat(t: torch.Tensor):
    """(ptr, rows, cols, pitch, dtype) of a 2-D tensor whose rows are contiguous."""
    r, c = t.shape
    if c > 1 and r > 0 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(-1) == 1)")
    ld = t.stride(0) if r > 1 else c
    if r > 1 and c > 0 and ld < c:
        raise ValueError("rows must not overlap (an expanded tensor needs .contiguous())")
    return _lib.MuonMat(t.data_ptr() or None, r, c, ld, _DT[t.dtype], 0)


def _array(kind, items):
    return (kind * len(items))(*items)


def _seed(opt_field: str, opt: "_lib.MXOptions", seed: Seed, device) -> None:
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != device:
            raise ValueError("a seed tensor holds one int64 on the operands' device")
        setattr(opt, opt_field + "_dev", seed.data_ptr())
    else:
        setattr(opt, opt_field, int(seed) & 0xFFFFFFFFFFFFFFFF)


def _same_device(items) -> torch.device:
    dev = items[0].device
    for t in items[1:]:
        if t.device != dev:
            raise ValueError("operands must be on one device")
    return dev


def _on(device):
    """Context that makes `device` current (free when it already is)."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _drop_options(opt, dropout: float, seed: Optional[Seed], device) -> None:
    if dropout:
        if seed is None:
            raise ValueError("dropout needs a seed")
        opt.dropout = float(dropout)
        _seed("dropout_seed", opt, seed, device)


def mx_quantize(x: Union[torch.Tensor, Sequence[torch.Tensor]], transpose: Union[bool, str] = False,
                seed: Optional[Seed] = None, dropout: float = 0.0,
                dropout_seed: Optional[Seed] = None, out=None):
    """x in 4 bits: an MX4 of x's rows (leading dimensions flattened), with
    transpose=True one of the transpose, with transpose="both" an MXPair of
    the two from one read.  Rounds to nearest, or stochastically with a
    `seed` (an int, or a one-element int64 tensor read when the kernel runs).
    `dropout` quantises what dropout(x, dropout, dropout_seed) would store.
    A list is quantised in one call and gives a list; `out` takes results of
    an earlier call of the same shapes and overwrites them."""
    if transpose not in (False, True, "both"):
        raise ValueError(f"transpose is False, True or 'both', not {transpose!r}")
    single = isinstance(x, torch.Tensor)
    xs = [_rows_of(t) for t in ([x] if single else x)]
    if not xs:
        return []
    dev = _same_device(xs)
    lib = _lib.load()
    both = transpose == "both"
    if out is None:
        rows = [MX4(t.shape[0], t.shape[1], dev) for t in xs] if transpose is not True else None
        cols = [MX4(t.shape[1], t.shape[0], dev) for t in xs] if transpose is not False else None
    else:
        outs = [out] if single else list(out)
        if len(outs) != len(xs):
            raise ValueError(f"{len(xs)} matrices, {len(outs)} outputs")
        rows = [o[0] if both else o for o in outs] if transpose is not True else None
        cols = [o[1] if both else o for o in outs] if transpose is not False else None
        _same_device(xs + (rows or []) + (cols or []))
    opt = _lib.MXOptions()
    if seed is not None:
        opt.stochastic = 1
        _seed("seed", opt, seed, dev)
    _drop_options(opt, dropout, dropout_seed, dev)
    with _on(dev):
        code = lib.muon_mx_quantize(_array(_lib.MuonMat, [_mat(t) for t in xs]),
                                    _array(_lib.MuonMX, [m.c for m in rows]) if rows else None,
                                    _array(_lib.MuonMX, [m.c for m in cols]) if cols else None,
                                    len(xs), opt, _stream(dev))
    _lib.check(code, "muon_mx_quantize")
    res = [MXPair(a, b) for a, b in zip(rows, cols)] if both else rows or cols
    return res[0] if single else res


def mx_dequantize(m: Union[MX4, Sequence[MX4]], dtype: torch.dtype = torch.bfloat16,
                  out: Union[None, torch.Tensor, Sequence[torch.Tensor]] = None):
    """The values that 4-bit matrices stand for, as rows x cols tensors."""
    single = isinstance(m, MX4)
    ms = [m] if single else list(m)
    if not ms:
        return []
    dev = _same_device(ms)
    if out is None:
        if dtype not in _DT:
            raise ValueError(f"unsupported dtype {dtype}")
        outs = [torch.empty(q.rows, q.cols, dtype=dtype, device=dev) for q in ms]
    else:
        outs = [_rows_of(t) for t in ([out] if single else out)]
        if len(outs) != len(ms):
            raise ValueError(f"{len(ms)} matrices, {len(outs)} outputs")
        _same_device(ms + outs)
    with _on(dev):
        code = _lib.load().muon_mx_dequantize(_array(_lib.MuonMX, [q.c for q in ms]),
                                              _array(_lib.MuonMat, [_mat(t) for t in outs]), len(ms),
                                              _stream(dev))
    _lib.check(code, "muon_mx_dequantize")
    return outs[0] if single else outs


def mx_matmul(a: Union[MX4, Sequence[MX4]], b: Union[MX4, Sequence[MX4]],
              dtype: torch.dtype = torch.bfloat16,
              out: Union[None, torch.Tensor, Sequence[torch.Tensor]] = None,
              accumulate: bool = False, dropout: float = 0.0, dropout_seed: Optional[Seed] = None):
    """a b^T of 4-bit matrices (both hold the contraction along their columns)
    with fp32 accumulation; lists are multiplied pairwise in one call.
    `accumulate` adds to `out`; `dropout` drops and scales the product's
    elements as dropout() does."""
    single = isinstance(a, MX4)
    la, lb = ([a], [b]) if single else (list(a), list(b))
    if len(la) != len(lb):
        raise ValueError(f"{len(la)} left and {len(lb)} right operands")
    if not la:
        return []
    dev = _same_device(la + lb)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if dtype not in _DT:
            raise ValueError(f"unsupported dtype {dtype}")
        outs = [torch.empty(p.rows, q.rows, dtype=dtype, device=dev) for p, q in zip(la, lb)]
    else:
        outs = [_rows_of(t) for t in ([out] if single else out)]
        if len(outs) != len(la):
            raise ValueError(f"{len(la)} products, {len(outs)} outputs")
        _same_device(la + outs)
    _matmul(la, lb, outs, dev, accumulate, dropout, dropout_seed)
    if out is not None:
        return out
    return outs[0] if single else outs


def _matmul(la, lb, outs, dev, accumulate=False, dropout=0.0, dropout_seed=None) -> None:
    opt = _lib.MXOptions()
    opt.accumulate = int(bool(accumulate))
    _drop_options(opt, dropout, dropout_seed, dev)
    with _on(dev):
        code = _lib.load().muon_mx_matmul(_array(_lib.MuonMX, [m.c for m in la]),
                                          _array(_lib.MuonMX, [m.c for m in lb]),
                                          _array(_lib.MuonMat, [_mat(t) for t in outs]), len(outs),
                                          opt, _stream(dev))
    _lib.check(code, "muon_mx_matmul")


def mx_linear(x: torch.Tensor, w: MX4, save: bool = False, dropout: float = 0.0,
              dropout_seed: Optional[Seed] = None):
    """x W^T for W in 4 bits and x [..., in] quantised here to nearest; the
    result [..., out] has x's type.  With `dropout` the layer's input is
    dropout(x, dropout, dropout_seed).  With `save` returns (y, saved), saved
    being what mx_linear_grad needs: the input's transpose in 4 bits."""
    x2 = _rows_of(x)
    if x2.shape[1] != w.cols:
        raise ValueError(f"x has {x2.shape[1]} features, the layer takes {w.cols}")
    q = mx_quantize(x2, "both" if save else False, dropout=dropout, dropout_seed=dropout_seed)
    y = mx_matmul(q[0] if save else q, w, dtype=x.dtype)
    y = y.view(*x.shape[:-1], w.rows)
    return (y, MXSaved(q[1], float(dropout), dropout_seed)) if save else y


def mx_linear_grad(dy: torch.Tensor, w_t: Optional[MX4], saved: MXSaved, seed: Optional[Seed] = None,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   grad_dtype: torch.dtype = torch.float32, pair: bool = False):
    """Gradients of mx_linear: (dx, dw) for the output gradient dy [..., out]
    and W^T in 4 bits (None: no dx).  dy is quantised once for both products,
    stochastically with a `seed`.  dw = dy^T x goes to a new tensor of
    grad_dtype or to `out` (added to it with `accumulate`); with `pair` its
    two 4-bit factors are returned instead, for Muon.step to multiply."""
    dy2 = _rows_of(dy)
    if dy2.shape[0] != saved.x_t.cols:
        raise ValueError(f"dy has {dy2.shape[0]} rows, the layer saw {saved.x_t.cols}")
    if w_t is not None and (w_t.cols != dy2.shape[1] or w_t.rows != saved.x_t.rows):
        raise ValueError(f"w_t is {w_t.rows} x {w_t.cols}, not {saved.x_t.rows} x {dy2.shape[1]}")
    q = mx_quantize(dy2, True if w_t is None else "both", seed=seed)
    dx = None
    dy_t = q
    if w_t is not None:
        dy_t = q[1]
        dx = mx_matmul(q[0], w_t, dtype=dy.dtype, dropout=saved.dropout,
                       dropout_seed=saved.dropout_seed).view(*dy.shape[:-1], w_t.rows)
    if pair:
        return dx, (dy_t, saved.x_t)
    return dx, mx_matmul(dy_t, saved.x_t, dtype=grad_dtype, out=out, accumulate=accumulate)


def dropout(x: torch.Tensor, p: float, seed: Seed, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with each element kept with probability 1 - p and scaled by
    1 / (1 - p), or zeroed; the same call on a gradient is the backward pass.
    `out` may be x itself."""
    x2 = _rows_of(x)
    res = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    if out is not None and out.shape != x.shape:
        raise ValueError(f"out is {tuple(out.shape)}, not {tuple(x.shape)}")
    o2 = _rows_of(res)
    dev = _same_device([x2, o2])
    opt = _lib.MXOptions()
    _seed("seed", opt, seed, dev)
    with _on(dev):
        code = _lib.load().muon_dropout(_mat(x2), _mat(o2), p, opt.seed, opt.seed_dev, _stream(dev))
    _lib.check(code, "muon_dropout")
    return res
