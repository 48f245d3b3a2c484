"""Tokens sorted by expert into a send buffer and back, with weights applied, and the gradients.

    rows, plan = dispatch(x, experts_of, num_experts)   # the buffer a compressed all-to-all takes
    out = combine(rows, weights, plan)                  # out[t] = sum_j weights[t, j] rows[position[t, j]]
    d_rows, d_weights = combine_grad(d_out, rows, weights, plan)
    dx = dispatch_grad(d_rows, plan)

``experts_of`` is [tokens, k] (int32 or int64); an id outside [0, num_experts) means no expert here (a dropped token,
or one that another rank holds): its row lies behind all experts' rows, holds zeros and adds nothing.  Values are
bfloat16, float16 or float32; sums are taken in float32, in slot order, and rounded once.  Tensors may have any row
stride.  Every call runs on ``stream`` (default: the current one) and does not synchronize.

Results have no autograd history: the gradients are the calls above.  A tensor that requires a gradient is refused while
gradients are recorded; use these calls under ``torch.no_grad``, on detached tensors or in a ``torch.autograd.Function``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._tensors import native, on


class Plan(NamedTuple):
    """Where each slot's row is: ``position`` int32 [tokens, k], and the first row of each expert, ``offsets`` int32
    [num_experts + 1] (rows from offsets[-1] on belong to no expert)."""

    position: torch.Tensor
    offsets: torch.Tensor

    @property
    def num_experts(self) -> int:
        return self.offsets.numel() - 1


def sort(experts_of, num_experts: int, stream=None) -> Plan:
    """The plan of a routing: the place of each slot in the order by expert, ties in slot order."""
    return Plan(*on(stream, (experts_of,), native.sort, experts_of, num_experts))


def dispatch(x, experts_of, num_experts: int, stream=None) -> tuple[torch.Tensor, Plan]:
    """x [tokens, hidden] as rows [tokens * k, hidden] sorted by expert, and the plan."""
    rows, position, offsets = on(stream, (experts_of, x), native.dispatch, x, experts_of, num_experts)
    return rows, Plan(position, offsets)


def dispatch_grad(d_rows, plan: Plan, stream=None) -> torch.Tensor:
    """The gradient of dispatch with respect to x: each token's sum of its rows' gradients."""
    return on(stream, (d_rows, *plan), native.combine, d_rows, None, *plan)


def combine(rows, weights, plan: Plan, stream=None) -> torch.Tensor:
    """Each token's rows [tokens * k, hidden] brought back and added with weights [tokens, k] (float32)."""
    if weights is None:
        raise TypeError("weights must be a CUDA tensor")
    return on(stream, (rows, weights, *plan), native.combine, rows, weights, *plan)


def combine_grad(d_out, rows, weights, plan: Plan, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients of combine with respect to rows and weights."""
    return on(stream, (d_out, rows, weights, *plan), native.combine_grad, d_out, rows, weights, *plan)
