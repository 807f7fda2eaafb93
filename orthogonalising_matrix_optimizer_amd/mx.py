"""4-bit operators and dropout: torch-facing wrappers of the C ABI.

Quantisation to microscaled 4-bit blocks, reading back, products over lists of
matrices, the linear layer with its gradients, and dropout whose mask is a
function of a seed and is never stored.  The number format and the random
numbers are stated in include/muon.h.  As in the rest of the package all
computation runs in the HIP library; this module allocates outputs and passes
pointers with the current stream of the tensors' device.  Descriptors are
packed as bytes: on a single token a call's cost is the host's.

A seed fixes the numbers of a call whatever layer it is for: give each layer
and each step its own (step * layers + layer), or all layers of a shape drop
the same elements.  Within a list each matrix has its own numbers.

Nothing here is recorded by autograd.  The gradients are calls of their own
(mx_linear_grad, dropout on the gradient), made by hand or by the two halves of
a torch.autograd.Function; mx_linear, mx_linear_grad and dropout refuse a tensor
that requires a gradient where autograd records.  mx_quantize takes weights
that require one.
"""
from __future__ import annotations

from ctypes import byref, c_int32
from functools import lru_cache
from math import prod
from struct import Struct
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.MUON_BF16, torch.float32: _lib.MUON_F32}
_MAT, _MX = "Pqqqii", "PPqq"      # muon_mat, muon_mx
_MAT1, _MX1 = Struct(_MAT), Struct(_MX)
_structs = lru_cache(maxsize=256)(lambda fields, n: Struct(fields * n))
_SPLIT = _lib.CODES["MUON_E_WORKSPACE"]

Seed = Union[int, torch.Tensor]


class MX4:
    """A rows x cols matrix in 4 bits (blocks of 32 along the columns share a scale).

    `data` holds codes and scales in the order in which the matrix
    instructions read them; use dequantize() for values.  The matrices that
    one call returns for a list share an allocation."""

    __slots__ = ("buffer", "offset", "device", "desc")

    def __init__(self, buffer: torch.Tensor, offset: int, device: torch.device,
                 desc: Tuple[int, int, int, int]):
        # desc: a muon_mx (codes, scales, rows, columns)
        self.buffer, self.offset, self.device, self.desc = buffer, offset, device, desc

    @property
    def rows(self) -> int:
        return self.desc[2]

    @property
    def cols(self) -> int:
        return self.desc[3]

    @property
    def shape(self) -> Tuple[int, int]:
        return self.desc[2:]

    @property
    def nbytes(self) -> int:
        return _mx_bytes(self.rows, self.cols)

    @property
    def data(self) -> torch.Tensor:
        return self.buffer[self.offset:self.offset + self.nbytes]

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
    (after dropout) and how to make the dropout mask again (of a seed tensor
    the value that the forward pass used)."""
    x_t: MX4
    dropout: float
    dropout_seed: Optional[Seed]


# Storage sizes (muon_mx_codes_bytes, muon_mx_scales_bytes): tiles of 16 x 128
# codes in 1024 bytes, of 64 x 128 elements' scales in 256.
def _mx_bytes(rows: int, cols: int) -> int:
    return (-(-rows // 16) * 1024 + -(-rows // 64) * 256) * -(-cols // 128)


_empty = torch.empty_strided      # 0.4 us less than torch.empty on the host


def _new_mx(rows, cols, device):
    """MX4 matrices of rows[i] x cols[i], in one allocation."""
    if len(rows) == 1:
        r, c = rows[0], cols[0]
        k, t = -(-c // 128), -(-r // 16) * 1024
        buf = _empty((k * (t + -(-r // 64) * 256),), (1,), dtype=torch.uint8, device=device)
        p = buf.data_ptr()
        return [MX4(buf, 0, device, (p, p + k * t, r, c) if p else (0, 0, r, c))]
    codes = [(r + 15 >> 4) * (c + 127 >> 7) << 10 for r, c in zip(rows, cols)]
    scales = [(r + 63 >> 6) * (c + 127 >> 7) << 8 for r, c in zip(rows, cols)]
    buf = torch.empty(sum(codes) + sum(scales), dtype=torch.uint8, device=device)
    p, at, out = buf.data_ptr(), 0, []
    for r, c, n, m in zip(rows, cols, codes, scales):
        q = p + at
        out.append(MX4(buf, at, device, (q, q + n, r, c) if n else (0, 0, r, c)))
        at += n + m
    return out


def _new_one(rows, cols, dtype, device):
    """A dense rows x cols tensor and its packed muon_mat."""
    d = _DT.get(dtype)
    if d is None:
        raise ValueError(f"unsupported dtype {dtype}")
    t = _empty((rows, cols), (cols or 1, 1), dtype=dtype, device=device)
    return t, _MAT1.pack(t.data_ptr(), rows, cols, cols, d, 0)


def _new_dense(rows, cols, dtype, device):
    """Dense rows[i] x cols[i] tensors and their packed muon_mat array; equally
    wide ones share an allocation."""
    n, width = len(rows), cols[0]
    if n == 1:
        t, mat = _new_one(rows[0], width, dtype, device)
        return [t], mat
    d = _DT.get(dtype)
    if d is None:
        raise ValueError(f"unsupported dtype {dtype}")
    if cols.count(width) == n:
        buf = torch.empty((sum(rows), width), dtype=dtype, device=device)
        p, step, flat = buf.data_ptr(), width * dtype.itemsize, []
        for r in rows:
            flat += (p, r, width, width, d, 0)
            p += r * step
        # nothing else refers to buf, so the parts need not be tied to it as views
        return list(torch.unsafe_split_with_sizes(buf, rows)), _structs(_MAT, n).pack(*flat)
    ts = [torch.empty(s, dtype=dtype, device=device) for s in zip(rows, cols)]
    return ts, _mats(ts, device)


def _rows_of(t: torch.Tensor) -> torch.Tensor:
    """`t` as a 2-D view of its rows (last dimension)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"expected a tensor, got {type(t).__name__}")
    n = t.dim()
    if n == 2:
        return t
    if n == 0:
        raise ValueError("tensors must have at least one dimension")
    c = t.shape[-1]
    try:
        return t.view(prod(t.shape[:-1]), c)
    except RuntimeError:
        raise ValueError("the leading dimensions must be one run of evenly spaced rows") from None


def _not_recorded(t: torch.Tensor) -> None:
    """Refuses a tensor whose gradient autograd would look for in the result."""
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError("the 4-bit operators and dropout record nothing for autograd: call them under "
                         "torch.no_grad() or in an autograd.Function, or give t.detach()")


def _written(ts) -> None:
    """Tells autograd that the library wrote tensors, as torch's own in-place operations do."""
    torch.autograd.graph.increment_version([t for t in ts if not t.is_inference()])


def _mat(t: torch.Tensor, dev: torch.device):
    """muon_mat of a 2-D tensor whose rows are contiguous."""
    d = _DT.get(t.dtype)
    if d is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if t.device != dev:
        raise ValueError("operands must be on one device" if t.is_cuda else "tensors must be on a GPU")
    r, c = t.shape
    s, one = t.stride()
    if r == 1 or c == 0:
        s = c
    elif s < c and r:
        raise ValueError("rows must not overlap (an expanded tensor needs .contiguous())")
    if one != 1 and c > 1 and r:
        raise ValueError("rows must be contiguous (stride(-1) == 1)")
    return t.data_ptr(), r, c, s, d, 0


def _flat(ts, dev):
    """The fields of the muon_mats of tensors' rows, one after the other."""
    flat, at, dt = [], dev.index, _DT
    for t in ts:
        # the usual operand without a call; any other is looked at in full
        if isinstance(t, torch.Tensor) and t.is_contiguous() and t.get_device() == at:
            s, d = t.shape, dt.get(t.dtype)
            if len(s) == 2 and d is not None:
                r, c = s
                flat += (t.data_ptr(), r, c, c, d, 0)
                continue
        flat += _mat(_rows_of(t), dev)
    return flat


def _mats(ts, dev) -> bytes:
    if len(ts) == 1:
        return _MAT1.pack(*_mat(ts[0], dev))
    return _structs(_MAT, len(ts)).pack(*_flat(ts, dev))


def _pack_mx(ms) -> bytes:
    if len(ms) == 1:
        return _MX1.pack(*ms[0].desc)
    flat = []
    for m in ms:
        flat += m.desc
    return _structs(_MX, len(ms)).pack(*flat)


def _mxs(ms, dev) -> bytes:
    for m in ms:
        if type(m) is not MX4:
            raise ValueError(f"expected an MX4, got {type(m).__name__}")
        if m.device is not dev and m.device != dev:
            raise ValueError("operands must be on one device")
    return _pack_mx(ms)


def _device_of(m) -> torch.device:
    if type(m) is not MX4:
        raise ValueError(f"expected an MX4, got {type(m).__name__}")
    return m.device


def _gpu(dev: torch.device) -> torch.device:
    if dev.index is None:        # a tensor on a GPU names which
        raise ValueError("tensors must be on a GPU")
    return dev


_functions = {}


def _call(name: str, dev: torch.device, *args) -> int:
    """A library call on `dev` and its current stream; raises on an error, but
    hands MUON_E_WORKSPACE back."""
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(_lib.load(), name)
    i = dev.index
    if _current_device() == i:
        code = f(*args, _current_stream(i))
    else:
        with torch.cuda.device(i):
            code = f(*args, _current_stream(i))
    if code and code != _SPLIT:
        _lib.check(code, name)
    return code


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _set_seed(opt: "_lib.MXOptions", field: str, seed: Seed, dev) -> None:
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != dev:
            raise ValueError("a seed tensor holds one int64 on the operands' device")
        setattr(opt, field + "_dev", seed.data_ptr())
    else:
        setattr(opt, field, int(seed) & 0xFFFFFFFFFFFFFFFF)


def _options(dev, seed: Optional[Seed] = None, dropout: float = 0.0,
             dropout_seed: Optional[Seed] = None, accumulate: bool = False):
    """muon_mx_options, or None for the defaults."""
    if seed is None and not dropout and not accumulate:
        return None
    opt = _lib.MXOptions()
    opt.accumulate = int(bool(accumulate))
    if seed is not None:
        opt.stochastic = 1
        _set_seed(opt, "seed", seed, dev)
    if dropout:
        if dropout_seed is None:
            raise ValueError("dropout needs a seed")
        opt.dropout = float(dropout)
        _set_seed(opt, "dropout_seed", dropout_seed, dev)
    return opt


def mx_quantize(x: Union[torch.Tensor, Sequence[torch.Tensor]], transpose: Union[bool, str] = False,
                seed: Optional[Seed] = None, dropout: float = 0.0,
                dropout_seed: Optional[Seed] = None, out=None):
    """x in 4 bits: an MX4 of x's rows (leading dimensions flattened), with
    transpose=True one of the transpose, with transpose="both" an MXPair of
    the two from one read.  Rounds to nearest, or stochastically with a
    `seed` (an int, or a one-element int64 tensor read when the kernel runs).
    `dropout` quantises what dropout(x, dropout, dropout_seed) would store (in
    a list, of its first matrix: each has the numbers of its place).
    A list is quantised in one call and gives a list; `out` takes results of
    an earlier call of the same shapes and overwrites them."""
    if transpose not in (False, True, "both"):
        raise ValueError(f"transpose is False, True or 'both', not {transpose!r}")
    both = transpose == "both"
    if not both:
        transpose = bool(transpose)      # 0, 1 and numpy's booleans pass the check above
    single = isinstance(x, torch.Tensor)
    xs = [x] if single else list(x)
    n = len(xs)
    if not xs:
        return []
    dev = _gpu(_rows_of(xs[0]).device)
    flat = _flat(xs, dev)
    mats = _MAT1.pack(*flat) if n == 1 else _structs(_MAT, n).pack(*flat)
    rows = cols = None
    if out is None:
        r, c = flat[1::6], flat[2::6]
        if transpose is not True:
            rows = _new_mx(r, c, dev)
        if transpose is not False:
            cols = _new_mx(c, r, dev)
    else:
        outs = [out] if single else list(out)
        if len(outs) != n:
            raise ValueError(f"{n} matrices, {len(outs)} outputs")
        if transpose is not True:
            rows = [o[0] if both else o for o in outs]
        if transpose is not False:
            cols = [o[1] if both else o for o in outs]
    opt = None
    if seed is not None or dropout:
        opt = _options(dev, seed, dropout, dropout_seed)
    pack = _pack_mx if out is None else lambda ms: _mxs(ms, dev)
    _call("muon_mx_quantize", dev, mats, pack(rows) if rows else None, pack(cols) if cols else None,
          n, opt)
    if both:
        res = [MXPair(a, b) for a, b in zip(rows, cols)]
    else:
        res = rows if rows else cols
    return res[0] if single else res


def quantize_again(xs: Sequence[torch.Tensor], pairs: Sequence[MXPair]):
    """The call mx_quantize(xs, "both", out=pairs) with its descriptors packed
    once, for a list that is quantised again and again in the same memory,
    which the returned function keeps alive."""
    dev = xs[0].device
    keep = list(xs), list(pairs)
    mats = _mats(xs, dev)
    rows, cols = _mxs([p.w for p in pairs], dev), _mxs([p.w_t for p in pairs], dev)

    def again() -> None:
        _call("muon_mx_quantize", dev, mats, rows, cols, len(keep[0]), None)
    return again


def mx_dequantize(m: Union[MX4, Sequence[MX4]], dtype: torch.dtype = torch.bfloat16,
                  out: Union[None, torch.Tensor, Sequence[torch.Tensor]] = None):
    """The values that 4-bit matrices stand for, as rows x cols tensors."""
    single = isinstance(m, MX4)
    ms = [m] if single else list(m)
    if not ms:
        return []
    dev = _device_of(ms[0])
    mxs = _mxs(ms, dev)
    if out is None:
        outs, mats = _new_dense([q.desc[2] for q in ms], [q.desc[3] for q in ms], dtype, dev)
    else:
        outs = [_rows_of(t) for t in ([out] if single else out)]
        if len(outs) != len(ms):
            raise ValueError(f"{len(ms)} matrices, {len(outs)} outputs")
        mats = _mats(outs, dev)
    _call("muon_mx_dequantize", dev, mxs, mats, len(ms))
    if out is not None:
        _written(outs)
        return out
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
    n = len(la)
    if n != len(lb):
        raise ValueError(f"{n} left and {len(lb)} right operands")
    if not la:
        return []
    dev = _device_of(la[0])
    ca, cb = _mxs(la, dev), _mxs(lb, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        outs, co = _new_dense([p.desc[2] for p in la], [q.desc[2] for q in lb], dtype, dev)
    else:
        outs = [_rows_of(t) for t in ([out] if single else out)]
        if len(outs) != n:
            raise ValueError(f"{n} products, {len(outs)} outputs")
        co = _mats(outs, dev)
    opt = _options(dev, None, dropout, dropout_seed, accumulate)
    code = _call("muon_mx_matmul", dev, ca, cb, co, n, opt, None, 0)
    if code == _SPLIT:   # the list's contraction is split: give it room for the partial products
        ws = torch.empty(int(_lib.load().muon_mx_matmul_workspace_bytes(ca, cb, n)), dtype=torch.uint8,
                         device=dev)
        _lib.check(_call("muon_mx_matmul", dev, ca, cb, co, n, opt, ws.data_ptr(), ws.numel()),
                   "muon_mx_matmul")
    if out is not None:
        _written(outs)
        return out
    return outs[0] if single else outs


def mx_plan_info(shapes: Sequence[Tuple[int, int, int]], dtype: torch.dtype = torch.bfloat16) -> dict:
    """How mx_matmul runs a list of M x N x K products (muon_mx_plan_info):
    the output tiles' height, the parts of each contraction, and of the first
    launch whether the outputs go past the caches and the XCDs' first items."""
    n = len(shapes)
    tile, past = c_int32(0), c_int32(0)
    parts, items = (c_int32 * n)(), (c_int32 * 9)()
    a, b, out = (_structs(fields, n).pack(*(v for s in shapes for v in f(*s))) for fields, f in (
        (_MX, lambda m, n, k: (0, 0, m, k)), (_MX, lambda m, n, k: (0, 0, n, k)),
        (_MAT, lambda m, n, k: (0, m, n, n, _DT[dtype], 0))))
    _lib.check(_lib.load().muon_mx_plan_info(a, b, out, n, byref(tile), parts, byref(past), items),
               "muon_mx_plan_info")
    return {"tile_rows": tile.value, "parts": list(parts), "past_caches": bool(past.value),
            "xcd_items": list(items)}


def mx_linear(x: torch.Tensor, w: MX4, save: bool = False, dropout: float = 0.0,
              dropout_seed: Optional[Seed] = None):
    """x W^T for W in 4 bits and x [..., in] quantised here to nearest; the
    result [..., out] has x's type.  With `dropout` the layer's input is
    dropout(x, dropout, dropout_seed), with a seed that no other layer or step
    has.  With `save` returns (y, saved), saved being what mx_linear_grad
    needs: the input's transpose in 4 bits."""
    _not_recorded(x)
    x2 = _rows_of(x)
    rows, cols = x2.shape
    _device_of(w)
    if cols != w.desc[3]:
        raise ValueError(f"x has {cols} features, the layer takes {w.cols}")
    if not save and not dropout and rows <= _lib.MX_FEW_ROWS and w.desc[2] <= _lib.MX_FEW_ROWS_MAX_N:
        dev = _gpu(x.device)
        xm = _MAT1.pack(*_mat(x2, dev))
        y, ym = _new_one(rows, w.desc[2], x.dtype, dev)
        _call("muon_mx_matmul_rows", dev, xm, _mxs([w], dev), ym)
        saved = None
    else:
        if save and dropout and isinstance(dropout_seed, torch.Tensor):
            # the backward pass needs this pass's value (a kernel also under capture)
            dropout_seed = dropout_seed + 0
        q = mx_quantize(x2, "both" if save else False, dropout=dropout, dropout_seed=dropout_seed)
        y = mx_matmul(q[0] if save else q, w, dtype=x.dtype)
        saved = MXSaved(q[1], float(dropout), dropout_seed) if save else None
    if x.dim() != 2:
        y = y.view(*x.shape[:-1], w.rows)
    return (y, saved) if save else y


def mx_linear_grad(dy: torch.Tensor, w_t: Optional[MX4], saved: MXSaved, seed: Optional[Seed] = None,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   grad_dtype: torch.dtype = torch.float32, pair: bool = False):
    """Gradients of mx_linear: (dx, dw) for the output gradient dy [..., out]
    and W^T in 4 bits (None: no dx).  dy is quantised once for both products,
    stochastically with a `seed`.  dw = dy^T x goes to a new tensor of
    grad_dtype or to `out` (added to it with `accumulate`); with `pair` its
    two 4-bit factors are returned instead, for Muon.step to multiply (then
    without out, accumulate and grad_dtype)."""
    if pair and (out is not None or accumulate or grad_dtype is not torch.float32):
        raise ValueError("pair=True returns factors: out, accumulate and grad_dtype have no use")
    _not_recorded(dy)
    dy2 = _rows_of(dy)
    if dy2.shape[0] != saved.x_t.cols:
        raise ValueError(f"dy has {dy2.shape[0]} rows, the layer saw {saved.x_t.cols}")
    if w_t is not None and (w_t.cols != dy2.shape[1] or w_t.rows != saved.x_t.rows):
        raise ValueError(f"w_t is {w_t.rows} x {w_t.cols}, not {saved.x_t.rows} x {dy2.shape[1]}")
    q = mx_quantize(dy2, True if w_t is None else "both", seed=seed)
    dx, dy_t = None, q
    if w_t is not None:
        dy_t = q[1]
        dx = mx_matmul(q[0], w_t, dtype=dy.dtype, dropout=saved.dropout,
                       dropout_seed=saved.dropout_seed)
        if dy.dim() != 2:
            dx = dx.view(*dy.shape[:-1], w_t.rows)
    if pair:
        return dx, (dy_t, saved.x_t)
    return dx, mx_matmul(dy_t, saved.x_t, dtype=grad_dtype, out=out, accumulate=accumulate)


def dropout(x: torch.Tensor, p: float, seed: Seed, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with each element kept with probability 1 - p and scaled by
    1 / (1 - p), or zeroed; the same call on a gradient is the backward pass.
    `out` may be x itself."""
    _not_recorded(x)
    x2 = _rows_of(x)
    dev = _gpu(x.device)
    xm = _MAT1.pack(*_mat(x2, dev))
    if out is None:
        res, om = _new_one(*x2.shape, x.dtype, dev)
        if x.dim() != 2:
            res = res.view(x.shape)
    else:
        if out.shape != x.shape:
            raise ValueError(f"out is {tuple(out.shape)}, not {tuple(x.shape)}")
        res, om = out, _MAT1.pack(*_mat(_rows_of(out), dev))
    if isinstance(seed, torch.Tensor):
        opt = _lib.MXOptions()
        _set_seed(opt, "seed", seed, dev)
        _call("muon_dropout", dev, xm, om, p, 0, opt.seed_dev)
    else:
        _call("muon_dropout", dev, xm, om, p, int(seed) & 0xFFFFFFFFFFFFFFFF, None)
    if out is not None:
        _written((out,))
    return res
