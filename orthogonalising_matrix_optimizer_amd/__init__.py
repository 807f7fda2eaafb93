"""MI355X (gfx950) Muon-style optimizer step: HIP kernels behind a C ABI.

`libmuon_mi355x.so` (built from csrc/ by `build.py`) does all the work; this
package only marshals torch tensors to its entry points.
"""
from . import _lib
from .optimizer import (CUBIC, QUINTIC, AdamW, Muon, StepGraph, coeff_rows, orthogonalize, plan_info,
                        probe_arm, probe_disarm, probe_read, workspace_bytes)
from .mx import (MX4, MXPair, MXSaved, dropout, mx_dequantize, mx_linear, mx_linear_grad, mx_matmul,
                 mx_plan_info, mx_quantize)
from .experts import (ExpertPlan, Routing, embedding, embedding_grad, expert_combine, expert_combine_grad,
                      expert_gather, expert_linear, expert_linear_grad, expert_plan, route, route_grad)

__all__ = ["Muon", "AdamW", "StepGraph", "orthogonalize", "workspace_bytes", "plan_info", "probe_arm",
           "probe_read", "probe_disarm", "coeff_rows", "CUBIC", "QUINTIC", "_lib",
           "MX4", "MXPair", "MXSaved", "mx_quantize", "mx_dequantize", "mx_matmul", "mx_linear",
           "mx_linear_grad", "mx_plan_info", "dropout",
           "ExpertPlan", "Routing", "route", "route_grad", "expert_plan", "expert_gather", "expert_linear",
           "expert_linear_grad", "expert_combine", "expert_combine_grad", "embedding", "embedding_grad"]
