"""Tokens sorted by expert into a send buffer and back, with weights applied, and the gradients.

    rows, plan = dispatch(x, experts_of, num_experts)   # the buffer a compressed all-to-all takes
    out = combine(rows, weights, plan)                  # out[t] = sum_j weights[t, j] rows[position[t, j]]
    d_rows, d_weights = combine_grad(d_out, rows, weights, plan)
    dx = dispatch_grad(d_rows, plan)

``experts_of`` is [tokens, k] (int32 or int64); an id outside [0, num_experts) means no expert here (a dropped token,
or one that another rank holds): its row lies behind all experts' rows, holds zeros and adds nothing.  Values are
bfloat16, float16 or float32; sums are taken in float32, in slot order, and rounded once.  Tensors may have any row
stride.  Every call runs on ``stream`` (default: the current one) and does not synchronize.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._tensors import MAX_EXPERTS, MAX_K, TYPES, call, check, current, fn, on, on_device, rows_of


class Plan(NamedTuple):
    """Where each slot's row is: ``position`` int32 [tokens, k], and the first row of each expert, ``offsets`` int32
    [num_experts + 1] (rows from offsets[-1] on belong to no expert)."""

    position: torch.Tensor
    offsets: torch.Tensor

    @property
    def num_experts(self) -> int:
        return self.offsets.numel() - 1


def _ids(experts_of, num_experts):
    on_device("experts_of", experts_of, (torch.int32, torch.int64), 2)
    check(1 <= num_experts <= MAX_EXPERTS, f"num_experts must be 1 to {MAX_EXPERTS}, got {num_experts}")
    check(1 <= experts_of.shape[1] <= MAX_K, f"experts_of must have 1 to {MAX_K} columns, got {experts_of.shape[1]}")


def _new_plan(ids, num_experts):
    slots, d = ids.numel(), ids.device
    workspace = torch.empty(fn("zc_moe_sort_workspace")(slots, num_experts), dtype=torch.uint8, device=d)
    return (Plan(torch.empty(ids.shape, dtype=torch.int32, device=d),
                 torch.empty(num_experts + 1, dtype=torch.int32, device=d)), workspace)


def _plan(plan):
    on_device("plan.position", plan.position, (torch.int32,), 2)
    on_device("plan.offsets", plan.offsets, (torch.int32,), 1)
    check(plan.position.is_contiguous() and plan.offsets.is_contiguous(), "a plan's tensors must be contiguous")
    check(2 <= plan.offsets.numel() <= MAX_EXPERTS + 1, f"a plan has 1 to {MAX_EXPERTS} experts")
    check(1 <= plan.position.shape[1] <= MAX_K, f"a plan has 1 to {MAX_K} slots a token")
    return plan.position.shape


def _rows(name, t, rows, like=None):
    on_device(name, t, tuple(TYPES) if like is None else (like.dtype,), 2)
    check(t.shape[0] == rows, f"{name} must have {rows} rows, got {t.shape[0]}")
    check(t.shape[1] >= 1 and (like is None or t.shape[1] == like.shape[1]), f"{name} has {t.shape[1]} columns")


def _weights(weights, plan):
    on_device("weights", weights, (torch.float32,), 2)
    check(weights.shape == plan.position.shape, f"weights must have the shape {tuple(plan.position.shape)}")


def sort(experts_of, num_experts: int, stream=None) -> Plan:
    """The plan of a routing: the place of each slot in the order by expert, ties in slot order."""
    _ids(experts_of, num_experts)
    with on(stream, experts_of):
        ids = experts_of.contiguous()
        plan, workspace = _new_plan(ids, num_experts)
        call("zc_moe_sort", ids.data_ptr(), ids.element_size(), ids.shape[0], ids.shape[1], num_experts,
             plan.position.data_ptr(), plan.offsets.data_ptr(), workspace.data_ptr(), current())
    return plan


def dispatch(x, experts_of, num_experts: int, stream=None) -> tuple[torch.Tensor, Plan]:
    """x [tokens, hidden] as rows [tokens * k, hidden] sorted by expert, and the plan."""
    _ids(experts_of, num_experts)
    tokens, k = experts_of.shape
    _rows("x", x, tokens)
    hidden = x.shape[1]
    with on(stream, experts_of, x):
        ids = experts_of.contiguous()
        x, pitch = rows_of(x)
        plan, workspace = _new_plan(ids, num_experts)
        rows = torch.empty((tokens * k, hidden), dtype=x.dtype, device=x.device)
        call("zc_moe_dispatch", x.data_ptr(), pitch, TYPES[x.dtype], ids.data_ptr(), ids.element_size(), tokens, k,
             num_experts, hidden, rows.data_ptr(), hidden, plan.position.data_ptr(), plan.offsets.data_ptr(),
             workspace.data_ptr(), current())
    return rows, plan


def _combine(rows, weights, plan, stream):
    tokens, k = _plan(plan)
    _rows("rows", rows, tokens * k)
    hidden = rows.shape[1]
    with on(stream, rows, weights, *plan):
        rows, pitch = rows_of(rows)
        weights = None if weights is None else weights.contiguous()
        out = torch.empty((tokens, hidden), dtype=rows.dtype, device=rows.device)
        call("zc_moe_combine", rows.data_ptr(), pitch, TYPES[rows.dtype], None if weights is None else weights.data_ptr(),
             plan.position.data_ptr(), plan.offsets.data_ptr(), tokens, k, plan.num_experts, hidden, out.data_ptr(),
             hidden, current())
    return out


def dispatch_grad(d_rows, plan: Plan, stream=None) -> torch.Tensor:
    """The gradient of dispatch with respect to x: each token's sum of its rows' gradients."""
    return _combine(d_rows, None, plan, stream)


def combine(rows, weights, plan: Plan, stream=None) -> torch.Tensor:
    """Each token's rows [tokens * k, hidden] brought back and added with weights [tokens, k] (float32)."""
    _plan(plan)
    _weights(weights, plan)
    return _combine(rows, weights, plan, stream)


def combine_grad(d_out, rows, weights, plan: Plan, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients of combine with respect to rows and weights."""
    tokens, k = _plan(plan)
    _weights(weights, plan)
    _rows("rows", rows, tokens * k)
    _rows("d_out", d_out, tokens, rows)
    hidden = rows.shape[1]
    with on(stream, rows, d_out, weights, *plan):
        rows, pitch = rows_of(rows)
        d_out, d_pitch = rows_of(d_out)
        weights = weights.contiguous()
        d_rows = torch.empty((tokens * k, hidden), dtype=rows.dtype, device=rows.device)
        d_weights = torch.empty((tokens, k), dtype=torch.float32, device=rows.device)
        call("zc_moe_combine_grad", d_out.data_ptr(), d_pitch, rows.data_ptr(), pitch, TYPES[rows.dtype],
             weights.data_ptr(), plan.position.data_ptr(), plan.offsets.data_ptr(), tokens, k, plan.num_experts,
             hidden, d_rows.data_ptr(), hidden, d_weights.data_ptr(), current())
    return d_rows, d_weights
