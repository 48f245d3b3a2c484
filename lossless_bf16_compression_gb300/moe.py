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

from ._tensors import MAX_EXPERTS, MAX_K, TYPES, call, current, fn, on, on_device, rows_of


class Plan(NamedTuple):
    """Where each slot's row is: ``position`` int32 [tokens, k], and the first row of each expert, ``offsets`` int32
    [num_experts + 1] (rows from offsets[-1] on belong to no expert)."""

    position: torch.Tensor
    offsets: torch.Tensor

    @property
    def num_experts(self) -> int:
        return self.offsets.numel() - 1


_ID_TYPES = (torch.int32, torch.int64)
_INT32 = (torch.int32,)
_FLOAT32 = (torch.float32,)
_ROW_TYPES = tuple(TYPES)


def _ids(experts_of, num_experts):
    device = on_device("experts_of", experts_of, None, _ID_TYPES, 2)
    if not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError(f"num_experts must be 1 to {MAX_EXPERTS}, got {num_experts}")
    if not 1 <= experts_of.shape[1] <= MAX_K:
        raise ValueError(f"experts_of must have 1 to {MAX_K} columns, got {experts_of.shape[1]}")
    return device


def _new_plan(ids, num_experts):
    need = fn("zc_moe_sort_workspace")(ids.numel(), num_experts)
    workspace = torch.empty(need, dtype=torch.uint8, device=ids.device) if need else None
    position = torch.empty_like(ids, dtype=torch.int32)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=ids.device)
    return Plan(position, offsets), None if workspace is None else workspace.data_ptr(), workspace


def _plan(plan):
    position, offsets = plan
    device = on_device("plan.position", position, None, _INT32, 2)
    on_device("plan.offsets", offsets, device, _INT32, 1)
    if not (position.is_contiguous() and offsets.is_contiguous()):
        raise ValueError("a plan's tensors must be contiguous")
    tokens, k = position.shape
    experts = offsets.shape[0] - 1
    if not (1 <= experts <= MAX_EXPERTS and 1 <= k <= MAX_K):
        raise ValueError(f"a plan has 1 to {MAX_EXPERTS} experts and 1 to {MAX_K} slots a token, got {experts} and {k}")
    return device, tokens, k, experts


def _rows(name, t, device, rows, dtypes=_ROW_TYPES, hidden=None):
    on_device(name, t, device, dtypes, 2)
    n, h = t.shape
    if n != rows or h < 1 or (hidden is not None and h != hidden):
        raise ValueError(f"{name} must be [{rows}, {'hidden' if hidden is None else hidden}], got {tuple(t.shape)}")
    return h


def _weights(weights, device, plan):
    on_device("weights", weights, device, _FLOAT32, 2)
    if weights.shape != plan[0].shape:
        raise ValueError(f"weights must have the shape {tuple(plan[0].shape)}, got {tuple(weights.shape)}")


def sort(experts_of, num_experts: int, stream=None) -> Plan:
    """The plan of a routing: the place of each slot in the order by expert, ties in slot order."""
    device = _ids(experts_of, num_experts)
    return on(stream, (experts_of,), _sort, experts_of, num_experts, device)


def _sort(ids, num_experts, device):
    ids = ids.contiguous()
    tokens, k = ids.shape
    plan, scratch, _keep = _new_plan(ids, num_experts)
    call("zc_moe_sort", ids.data_ptr(), ids.element_size(), tokens, k, num_experts, plan[0].data_ptr(),
         plan[1].data_ptr(), scratch, current(device))
    return plan


def dispatch(x, experts_of, num_experts: int, stream=None) -> tuple[torch.Tensor, Plan]:
    """x [tokens, hidden] as rows [tokens * k, hidden] sorted by expert, and the plan."""
    device = _ids(experts_of, num_experts)
    hidden = _rows("x", x, device, experts_of.shape[0])
    return on(stream, (experts_of, x), _dispatch, x, experts_of, num_experts, hidden, device)


def _dispatch(x, ids, num_experts, hidden, device):
    ids = ids.contiguous()
    tokens, k = ids.shape
    x, pitch = rows_of(x)
    plan, scratch, _keep = _new_plan(ids, num_experts)
    rows = torch.empty((tokens * k, hidden), dtype=x.dtype, device=x.device)
    call("zc_moe_dispatch", x.data_ptr(), pitch, TYPES[x.dtype], ids.data_ptr(), ids.element_size(), tokens, k,
         num_experts, hidden, rows.data_ptr(), hidden, plan[0].data_ptr(), plan[1].data_ptr(), scratch,
         current(device))
    return rows, plan


def _combine(rows, weights, plan, shape):
    device, tokens, k, experts, hidden = shape
    rows, pitch = rows_of(rows)
    if weights is not None:
        weights = weights.contiguous()
    out = torch.empty((tokens, hidden), dtype=rows.dtype, device=rows.device)
    call("zc_moe_combine", rows.data_ptr(), pitch, TYPES[rows.dtype], None if weights is None else weights.data_ptr(),
         plan[0].data_ptr(), plan[1].data_ptr(), tokens, k, experts, hidden, out.data_ptr(), hidden, current(device))
    return out


def dispatch_grad(d_rows, plan: Plan, stream=None) -> torch.Tensor:
    """The gradient of dispatch with respect to x: each token's sum of its rows' gradients."""
    device, tokens, k, experts = _plan(plan)
    hidden = _rows("d_rows", d_rows, device, tokens * k)
    return on(stream, (d_rows, *plan), _combine, d_rows, None, plan, (device, tokens, k, experts, hidden))


def combine(rows, weights, plan: Plan, stream=None) -> torch.Tensor:
    """Each token's rows [tokens * k, hidden] brought back and added with weights [tokens, k] (float32)."""
    device, tokens, k, experts = _plan(plan)
    hidden = _rows("rows", rows, device, tokens * k)
    _weights(weights, device, plan)
    return on(stream, (rows, weights, *plan), _combine, rows, weights, plan, (device, tokens, k, experts, hidden))


def combine_grad(d_out, rows, weights, plan: Plan, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients of combine with respect to rows and weights."""
    device, tokens, k, experts = _plan(plan)
    _weights(weights, device, plan)
    hidden = _rows("rows", rows, device, tokens * k)
    _rows("d_out", d_out, device, tokens, (rows.dtype,), hidden)
    return on(stream, (d_out, rows, weights, *plan), _combine_grad, d_out, rows, weights, plan,
              (device, tokens, k, experts, hidden))


def _combine_grad(d_out, rows, weights, plan, shape):
    device, tokens, k, experts, hidden = shape
    rows, pitch = rows_of(rows)
    d_out, d_pitch = rows_of(d_out)
    weights = weights.contiguous()
    d_rows = torch.empty((tokens * k, hidden), dtype=rows.dtype, device=rows.device)
    d_weights = torch.empty_like(weights)
    call("zc_moe_combine_grad", d_out.data_ptr(), d_pitch, rows.data_ptr(), pitch, TYPES[rows.dtype],
         weights.data_ptr(), plan[0].data_ptr(), plan[1].data_ptr(), tokens, k, experts, hidden, d_rows.data_ptr(),
         hidden, d_weights.data_ptr(), current(device))
    return d_rows, d_weights
