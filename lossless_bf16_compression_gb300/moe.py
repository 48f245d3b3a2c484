"""A router's choice of experts, tokens sorted by expert into a send buffer and back with weights applied, and the gradients.

    weights, experts_of = route(logits, k)              # the k largest of each token's logits, and their scores
    loss, counts, slope = balance(logits, experts_of)   # the loss that keeps experts evenly used, and their slots
    d_logits = route_grad(d_weights, logits, experts_of, balance=(d_loss, Balance(loss, counts, slope)))

    rows, plan = dispatch(x, experts_of, num_experts)   # the buffer a compressed all-to-all takes
    out = combine(rows, weights, plan)                  # out[t] = sum_j weights[t, j] rows[position[t, j]]
    d_rows, d_weights = combine_grad(d_out, rows, weights, plan)
    dx = dispatch_grad(d_rows, plan)

``experts_of`` is [tokens, k] (int32 or int64); an id outside [0, num_experts) means no expert here (a dropped token,
or one that another rank holds): its row lies behind all experts' rows, holds zeros and adds nothing.  Values are
bfloat16, float16 or float32; sums are taken in float32, in slot order, and rounded once.  Tensors may have any row
stride.  Every call runs on ``stream`` (default: the current one) and does not synchronize.

``logits`` are [tokens, experts], of any of these types; a logit of -infinity means that a token may not use an expert, and
a row of nothing but -infinity is padding.  ``score`` is "softmax" (of the row) or "sigmoid" (of each logit).

Results have no autograd history: the gradients are the calls above.  A tensor that requires a gradient is refused while
gradients are recorded; use these calls under ``torch.no_grad``, on detached tensors or in a ``torch.autograd.Function``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._tensors import native, on


SCORES = {"softmax": 0, "sigmoid": 1}


class Balance(NamedTuple):
    """The balance loss (float32, 0 dimensions), each expert's slots ``counts`` (int32 [experts]), and the loss's derivative
    in any token's probability of each expert, ``slope`` (float32 [experts])."""

    loss: torch.Tensor
    counts: torch.Tensor
    slope: torch.Tensor


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


def _score(score):
    s = SCORES.get(score)
    if s is None:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, got {score!r}")
    return s


def route(logits, k: int, score: str = "softmax", normalize: bool = True, scale: float = 1.0,
          stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Each token's k largest logits, largest first, equal ones by expert: (weights float32 [tokens, k], experts_of int32
    [tokens, k]).

    A weight is ``scale`` times the expert's score, with ``normalize`` divided by the sum of the token's chosen ones.
    -infinity is never chosen: where fewer than k logits are left, the other slots get the id -1 (no expert, for
    dispatch) and the weight 0.  A NaN counts as larger than every number and shows in the weights."""
    return on(stream, (logits,), native.route, logits, k, _score(score), bool(normalize), scale)


def balance(logits, experts_of, score: str = "softmax", stream=None) -> Balance:
    """The loss experts / (k n^2) * sum_e counts[e] * sum_t p[t, e] of a routing, 1 when all experts are used alike.

    p is the softmax of a row, or its sigmoids divided by their sum; n counts the rows that are not padding; counts[e] are
    the slots of ``experts_of`` [tokens, k] (int32) that hold e (ids outside the experts are in none)."""
    return Balance(*on(stream, (logits, experts_of), native.balance, logits, experts_of, _score(score)))


def balance_grad(d_loss, logits, balance: Balance, score: str = "softmax", stream=None) -> torch.Tensor:
    """The gradient of the balance loss with respect to the logits; ``d_loss`` is a float32 tensor of one element."""
    if d_loss is None:
        raise TypeError("d_loss must be a CUDA tensor")
    slope = balance.slope
    return on(stream, (d_loss, logits, slope), native.route_grad, logits, None, None, d_loss, slope, _score(score), True, 1.0)


def route_grad(d_weights, logits, experts_of, score: str = "softmax", normalize: bool = True, scale: float = 1.0,
               balance: tuple[torch.Tensor, Balance] | None = None, stream=None) -> torch.Tensor:
    """The gradient of route's weights with respect to the logits, of the logits' type.

    ``score``, ``normalize``, ``scale`` and ``experts_of`` are those of the forward call; slots without an expert, or with one whose
    logit is -infinity, add nothing, whatever their ``d_weights``.  With ``balance`` = (d_loss, what
    balance returned for the same score), that loss's gradient is added before the one rounding."""
    if d_weights is None or experts_of is None:
        raise TypeError("d_weights and experts_of must be CUDA tensors")
    d_loss, slope = (None, None) if balance is None else (balance[0], balance[1].slope)
    if balance is not None and d_loss is None:
        raise TypeError("d_loss must be a CUDA tensor")
    return on(stream, (d_weights, logits, experts_of, d_loss, slope), native.route_grad, logits, d_weights, experts_of,
              d_loss, slope, _score(score), bool(normalize), scale)
