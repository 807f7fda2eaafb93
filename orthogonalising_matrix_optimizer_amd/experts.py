"""Layers of experts and the embedding table: torch-facing wrappers of the C ABI.

`route` chooses each token's experts and sorts the tokens by expert;
`expert_linear` multiplies the sorted rows with their experts' matrices, whose
gradients (`expert_linear_grad`) Muon.step takes; `expert_combine` sums the
experts' rows back to tokens; `embedding` looks tokens up in a table, whose
gradient AdamW.step takes.  The number of rows of each expert stays on the
device: no call waits for the GPU, and all may be captured into a graph.

Nothing here is recorded by autograd.  As for the 4-bit layers the gradients are
calls of their own, made by hand or by the two halves of a
torch.autograd.Function, and a tensor (an output's too) that requires a gradient
is refused where autograd records, one with a tangent of forward mode always.
"""
from __future__ import annotations

from struct import Struct
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .mx import _DT, _MAT1, _call, _empty, _gpu, _mat, _new_one, _not_recorded, _rows_of, _written

_SLOTS, _STACK, _IDS = Struct("PPPqii"), Struct("Pqqqqqii"), Struct("Pqii")
_I32 = torch.int32


class ExpertPlan:
    """The slots (token t, choice j) of a choice of experts, sorted by expert, by
    slot among equals: rows offsets[e] to offsets[e + 1] - 1 belong to expert e.

    offsets [experts + 1], tokens [slots] (each row's token, -1 behind the last
    expert's rows) and place [tokens, k] (each slot's row, -1 if its expert was
    none of 0 .. experts - 1) are int32 tensors on the device."""

    __slots__ = ("buffer", "n_tokens", "k", "experts", "device", "desc")

    def __init__(self, buffer: torch.Tensor, n_tokens: int, k: int, experts: int, device: torch.device,
                 _own: bool = False):
        # buffer: place, tokens and offsets, int32 (_own: allocated for them)
        if not _own:
            _check_counts(n_tokens, k, experts)
            n = 2 * n_tokens * k + experts + 1
            if not isinstance(buffer, torch.Tensor) or buffer.dtype != _I32 or buffer.device != device or \
                    buffer.dim() != 1 or not buffer.is_contiguous() or buffer.storage_offset() or buffer.numel() < n:
                raise ValueError(f"a plan of {n_tokens} tokens x {k} and {experts} experts is a tensor of {n} int32 "
                                 f"on {device}, from its memory's start")
        self.buffer, self.n_tokens, self.k, self.experts, self.device = buffer, n_tokens, k, experts, device
        p, n = buffer.data_ptr(), 4 * n_tokens * k
        self.desc = _SLOTS.pack(p + 2 * n, p + n, p, n_tokens, k, experts)

    @property
    def offsets(self) -> torch.Tensor:
        return self.buffer.as_strided((self.experts + 1,), (1,), 2 * self.slots)

    @property
    def tokens(self) -> torch.Tensor:
        return self.buffer.as_strided((self.slots,), (1,), self.slots)

    @property
    def place(self) -> torch.Tensor:
        return self.buffer.as_strided((self.n_tokens, self.k), (self.k, 1), 0)

    @property
    def slots(self) -> int:
        return self.n_tokens * self.k

    def __repr__(self) -> str:
        return f"ExpertPlan({self.n_tokens} tokens x {self.k}, {self.experts} experts, {self.device})"


class Routing(NamedTuple):
    """gates [tokens, k] fp32, experts [tokens, k] int32 (-1: none), their
    sorted slots, and whether the gates are normalised over the chosen."""
    gates: torch.Tensor
    experts: torch.Tensor
    plan: ExpertPlan
    normalize: bool


def _workspace(n: int, dev: torch.device):
    """Scratch memory of n bytes (or none), its address and size."""
    if not n:
        return None, None, 0
    t = _empty((n,), (1,), dtype=torch.uint8, device=dev)
    return t, t.data_ptr(), n


def _check_counts(n_tokens: int, k: int, experts: int) -> None:
    if not 1 <= experts <= _lib.MAX_EXPERTS:
        raise ValueError(f"1 to {_lib.MAX_EXPERTS} experts, not {experts}")
    if not 1 <= k <= _lib.MAX_K:
        raise ValueError(f"1 to {_lib.MAX_K} experts a token, not {k}")
    if not 0 <= n_tokens * k <= _lib.MAX_SLOTS:
        raise ValueError(f"{n_tokens} tokens x {k} are not 0 to {_lib.MAX_SLOTS} slots")


def _ids(t: torch.Tensor, dev: Optional[torch.device] = None) -> Tuple[torch.Tensor, bytes]:
    """Integers in one run (t, or a copy of rows that are apart) and their muon_ids."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"expected a tensor, got {type(t).__name__}")
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"indexes are int32 or int64, not {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError("operands must be on one device")
    if not t.is_contiguous():
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("rows of indexes must be contiguous (stride(-1) == 1)")
        t = t.contiguous()
    return t, _IDS.pack(t.data_ptr(), t.numel(), t.element_size(), 0)


def _per_slot(t: torch.Tensor, plan_shape: Tuple[int, int], dev: torch.device, what: str,
              dtype: torch.dtype = torch.float32) -> int:
    """The address of a dense tensor (fp32 or of `dtype`) with one number a slot."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev:
        raise ValueError(f"{what} must be a tensor of {dtype} on the operands' device")
    if tuple(t.shape) != plan_shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and {plan_shape[0]} x {plan_shape[1]}, not {tuple(t.shape)}")
    return t.data_ptr()


def _stack(w: torch.Tensor, dev: torch.device) -> bytes:
    """muon_stack of a 3-D tensor whose matrices' rows are contiguous."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("the experts' matrices are one 3-D tensor [experts, out, in]")
    d = _DT.get(w.dtype)
    if d is None:
        raise ValueError(f"unsupported dtype {w.dtype}")
    if w.device != dev:
        raise ValueError("operands must be on one device")
    n, r, c = w.shape
    s, ld, one = w.stride()
    if one != 1 and c > 1 and n * r:
        raise ValueError("rows must be contiguous (stride(-1) == 1)")
    if r <= 1 or c == 0:
        ld = c
    if n <= 1 or r * c == 0:
        s = r * ld
    if ld < c or s < (r - 1) * ld + c and r * c:
        raise ValueError("matrices and their rows must not overlap (an expanded tensor needs .contiguous())")
    return _STACK.pack(w.data_ptr(), n, r, c, ld, s, d, 0)


def _rows_mat(t: torch.Tensor, rows: int, dev: torch.device, what: str) -> bytes:
    """muon_mat of a 2-D tensor of `rows` rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    if t.shape[0] != rows:
        raise ValueError(f"{what} has {t.shape[0]} rows, not {rows}")
    return _MAT1.pack(*_mat(t, dev))


def _result(out: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype, dev: torch.device):
    """`out` or a new tensor, and its packed muon_mat."""
    if out is None:
        return _new_one(rows, cols, dtype, dev)
    _not_recorded(out)
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"out is {tuple(out.shape)}, not {(rows, cols)}")
    return out, _MAT1.pack(*_mat(out, dev))


def _plan_of(plan: ExpertPlan) -> torch.device:
    if type(plan) is not ExpertPlan:
        raise ValueError(f"expected an ExpertPlan, got {type(plan).__name__}")
    return plan.device


def expert_plan(experts: torch.Tensor, n_experts: int) -> ExpertPlan:
    """Sorts the slots of a choice of experts [tokens, k] (int32 or int64, rows
    contiguous; a number outside 0 .. n_experts - 1 drops its slot), for routers other
    than route()."""
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise ValueError("the choice of experts is a 2-D tensor [tokens, k]")
    dev = _gpu(experts.device)
    n, k = experts.shape
    _check_counts(n, k, n_experts)
    held, ids = _ids(experts)
    plan = ExpertPlan(_empty((2 * n * k + n_experts + 1,), (1,), dtype=_I32, device=dev), n, k, n_experts, dev, True)
    keep, ws, size = _workspace(int(_lib.load().muon_expert_plan_workspace_bytes(n, k, n_experts)), dev)
    _lib.check(_call("muon_expert_plan", dev, ids, plan.desc, ws, size), "muon_expert_plan")
    return plan


def route(logits: torch.Tensor, k: int, normalize: bool = False) -> Routing:
    """The k experts with the largest logits [tokens, experts] of each token
    (ties to the lowest), their gates (softmax over all experts, or with
    `normalize` over the chosen) and their sorted slots.  An expert with the
    logit -inf is never chosen; where none is left a slot has expert -1 and gate
    0, so a token of padding is one whose logits are all -inf."""
    _not_recorded(logits)
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits are a 2-D tensor [tokens, experts]")
    dev = _gpu(logits.device)
    n, e = logits.shape
    k = int(k)
    _check_counts(n, k, e)
    mat = _MAT1.pack(*_mat(logits, dev))
    # one allocation: the plan, then the chosen experts and the gates
    m = n * k
    buf = _empty((4 * m + e + 1,), (1,), dtype=_I32, device=dev)
    plan = ExpertPlan(buf, n, k, e, dev, True)
    at = 2 * m + e + 1
    chosen = buf.as_strided((n, k), (k, 1), at)
    gates = buf.view(torch.float32).as_strided((n, k), (k, 1), at + m)
    p = buf.data_ptr() + 4 * at
    keep, ws, size = _workspace(int(_lib.load().muon_expert_plan_workspace_bytes(n, k, e)), dev)
    _lib.check(_call("muon_route", dev, mat, int(bool(normalize)), p + 4 * m, p, plan.desc, ws, size), "muon_route")
    return Routing(gates, chosen, plan, bool(normalize))


def route_grad(dgates: torch.Tensor, logits: torch.Tensor, routing: Routing) -> torch.Tensor:
    """Gradient of routing.gates with respect to the logits, in their type.  A
    Routing of a router of one's own has fp32 gates and int32 experts [tokens, k],
    both contiguous, and expert_plan's plan of them."""
    if not isinstance(routing, Routing) or type(routing.plan) is not ExpertPlan:
        raise ValueError("routing is a Routing with an ExpertPlan")
    _not_recorded(dgates, logits, routing.gates)
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits are a 2-D tensor [tokens, experts]")
    dev = _gpu(logits.device)
    n, e = logits.shape
    plan = routing.plan
    shape = (plan.n_tokens, plan.k)
    if shape[0] != n or plan.experts != e:
        raise ValueError(f"logits are {n} x {e}, the routing of {shape[0]} tokens and {plan.experts} experts")
    dg, g = _per_slot(dgates, shape, dev, "dgates"), _per_slot(routing.gates, shape, dev, "routing.gates")
    chosen = _per_slot(routing.experts, shape, dev, "routing.experts", _I32)
    out, om = _new_one(n, e, logits.dtype, dev)
    _call("muon_route_grad", dev, dg, _MAT1.pack(*_mat(logits, dev)), g, chosen, plan.k, int(bool(routing.normalize)),
          om)
    return out


def expert_gather(x: torch.Tensor, plan: ExpertPlan, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The tokens' rows [tokens, cols] in the order of the plan's rows.  Rows
    that belong to no slot are left as they were."""
    _not_recorded(x)
    dev = _plan_of(plan)
    xm = _rows_mat(x, plan.n_tokens, dev, "x")
    res, om = _result(out, plan.slots, x.shape[1], x.dtype, dev)
    _call("muon_expert_gather", dev, xm, plan.desc, om)
    if out is not None:
        _written((out,))
    return res


def _sorted_rows(x: torch.Tensor, plan: ExpertPlan, gather: bool, dev: torch.device):
    """x, its muon_mat and whether the product gathers it: rows of tokens
    that span more than a product can address are gathered first."""
    if gather and isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[0] > 1 and \
            ((x.shape[0] - 1) * x.stride(0) + x.shape[1]) * x.element_size() >= _lib.GATHER_BYTES:
        x, gather = expert_gather(x, plan), False
    return x, _rows_mat(x, plan.n_tokens if gather else plan.slots, dev, "x"), gather


def expert_linear(x: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, gather: bool = False,
                  out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Each row of x times its expert's matrix: x[r] w[e]^T for w [experts, out,
    in], [slots, out] in x's type or `dtype`.  x [slots, in] is in the order of the
    plan's rows, or with `gather` [tokens, in], one row a token.  Rows that
    belong to no slot are left as they were (uninitialised without `out`).  fp32
    operands keep their 24 bits; one of 3.3895e38 or more counts as an infinity."""
    _not_recorded(x, w)
    dev = _plan_of(plan)
    wm = _stack(w, dev)
    x, xm, gather = _sorted_rows(x, plan, gather, dev)
    if x.shape[1] != w.shape[2] or w.shape[0] != plan.experts:
        raise ValueError(f"x has {x.shape[1]} features and the plan {plan.experts} experts, the matrices are "
                         f"{tuple(w.shape)}")
    res, om = _result(out, plan.slots, w.shape[1], dtype or x.dtype, dev)
    _call("muon_expert_linear", dev, xm, wm, plan.desc, int(gather), om)
    if out is not None:
        _written((out,))
    return res


def expert_linear_grad(dy: torch.Tensor, w: Optional[torch.Tensor], x: Optional[torch.Tensor], plan: ExpertPlan,
                       gather: bool = False, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       grad_dtype: torch.dtype = torch.float32):
    """Gradients of expert_linear: (dx, dw) for the output gradient dy [slots,
    out].  dx [slots, in] has dy's type and a row for each slot also where the
    layer gathered: expert_combine(dx, plan) sums them to tokens.  dw [experts,
    out, in] goes to a new tensor of grad_dtype or to `out` (added to it with
    `accumulate`); list(dw) are gradients for Muon.step.  Without w there is no
    dx, without x no dw."""
    _not_recorded(dy, w, x, out)
    dev = _plan_of(plan)
    dm = _rows_mat(dy, plan.slots, dev, "dy")
    dx = dw = None
    if w is not None:
        wm = _stack(w, dev)
        if w.shape[1] != dy.shape[1] or w.shape[0] != plan.experts:
            raise ValueError(f"dy has {dy.shape[1]} features and the plan {plan.experts} experts, the matrices are "
                             f"{tuple(w.shape)}")
        if x is not None and x.shape[-1] != w.shape[2]:
            raise ValueError(f"x has {x.shape[-1]} features, the matrices are {tuple(w.shape)}")
    if x is None and (out is not None or accumulate):
        raise ValueError("out and accumulate are for dw, which needs x")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if x is not None:
        x, xm, gather = _sorted_rows(x, plan, gather, dev)
        shape = (plan.experts, dy.shape[1], x.shape[1])
        if out is None:
            if grad_dtype not in _DT:
                raise ValueError(f"unsupported dtype {grad_dtype}")
            dw = torch.empty(shape, dtype=grad_dtype, device=dev)
        elif tuple(out.shape) != shape:
            raise ValueError(f"out is {tuple(out.shape)}, not {shape}")
        else:
            dw = out
        dwm = _stack(dw, dev)
    if w is not None:
        dx, dxm = _new_one(plan.slots, w.shape[2], dy.dtype, dev)
        _call("muon_expert_linear_dx", dev, dm, wm, plan.desc, dxm)
    if x is not None:
        keep, ws, size = _workspace(int(_lib.load().muon_expert_linear_dw_workspace_bytes(plan.slots, dwm)), dev)
        _lib.check(_call("muon_expert_linear_dw", dev, dm, xm, plan.desc, int(gather), int(bool(accumulate)), dwm,
                         ws, size), "muon_expert_linear_dw")
        if out is not None:
            _written((out,))
    return dx, dw


def expert_combine(y: torch.Tensor, plan: ExpertPlan, gates: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The rows y [slots, cols] of each token's slots summed, each times its gate
    [tokens, k] (fp32; None: ones, the gradient of gathered rows): [tokens,
    cols] in y's type or `dtype`, zeros for a token without slots."""
    _not_recorded(y, gates)
    dev = _plan_of(plan)
    ym = _rows_mat(y, plan.slots, dev, "y")
    g = None if gates is None else _per_slot(gates, (plan.n_tokens, plan.k), dev, "gates")
    res, om = _result(out, plan.n_tokens, y.shape[1], dtype or y.dtype, dev)
    _call("muon_expert_combine", dev, ym, g, plan.desc, om)
    if out is not None:
        _written((out,))
    return res


def expert_combine_grad(dout: torch.Tensor, y: torch.Tensor, plan: ExpertPlan,
                        gates: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of expert_combine: (dy [slots, cols] in dout's type, dgates
    [tokens, k] in fp32, 0 for dropped slots).  Rows of dy that belong to no
    slot are uninitialised."""
    _not_recorded(dout, y, gates)
    dev = _plan_of(plan)
    dm = _rows_mat(dout, plan.n_tokens, dev, "dout")
    ym = _rows_mat(y, plan.slots, dev, "y")
    if y.shape[1] != dout.shape[1]:
        raise ValueError(f"dout has {dout.shape[1]} features, y {y.shape[1]}")
    g = _per_slot(gates, (plan.n_tokens, plan.k), dev, "gates")
    dy, dym = _new_one(plan.slots, dout.shape[1], dout.dtype, dev)
    dgates = _empty((plan.n_tokens, plan.k), (plan.k, 1), dtype=torch.float32, device=dev)
    _call("muon_expert_combine_grad", dev, dm, ym, g, plan.desc, dym, dgates.data_ptr())
    return dy, dgates


def embedding(ids: torch.Tensor, w: torch.Tensor, scale: float = 1.0,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale times the rows of the table w [rows, cols] that ids (int32 or int64,
    any shape, rows contiguous: tokens[:, :-1], say) name: [*ids.shape, cols] in w's
    type.  An id that is none of w's rows (-1, say: padding) gives zeros."""
    _not_recorded(w)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("the table is a 2-D tensor [rows, cols]")
    dev = _gpu(w.device)
    (held, im), wm = _ids(ids, dev), _MAT1.pack(*_mat(w, dev))
    shape = (*ids.shape, w.shape[1])
    if out is None:
        res, om = _new_one(ids.numel(), w.shape[1], w.dtype, dev)
        if len(shape) != 2:
            res = res.view(shape)
    else:
        _not_recorded(out)
        if tuple(out.shape) != shape:
            raise ValueError(f"out is {tuple(out.shape)}, not {shape}")
        res, om = out, _MAT1.pack(*_mat(_rows_of(out), dev))
    _call("muon_embedding", dev, im, wm, float(scale), om)
    if out is not None:
        _written((out,))
    return res


def embedding_grad(dy: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   grad_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Gradient of embedding with respect to its table of `rows` rows: scale
    times the sums of dy [*ids.shape, cols] over the places of each id, in a
    new tensor of grad_dtype or in `out` (added to it with `accumulate`)."""
    _not_recorded(dy)
    if tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"dy is {tuple(dy.shape)}, ids are {tuple(ids.shape)}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    d2 = _rows_of(dy)
    dev = _gpu(dy.device)
    dm, (held, im) = _MAT1.pack(*_mat(d2, dev)), _ids(ids, dev)
    rows, cols = int(rows), d2.shape[1]
    res, om = _result(out, rows, cols, grad_dtype, dev)
    keep, ws, size = _workspace(int(_lib.load().muon_embedding_grad_workspace_bytes(ids.numel(), rows, cols)), dev)
    _lib.check(_call("muon_embedding_grad", dev, dm, im, float(scale), int(bool(accumulate)), om, ws, size),
               "muon_embedding_grad")
    if out is not None:
        _written((out,))
    return res
