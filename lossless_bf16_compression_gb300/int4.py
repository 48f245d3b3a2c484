"""Weights in 4 bits with a scale for each group of 128, and the experts' products on them, for decoding.

    w = quantize_weight(weight)                # [experts, n, k] or [n, k]
    y = matmul(x, w, offsets)                  # rows offsets[e] .. offsets[e + 1] - 1 times expert e's w^T

``offsets`` is int32 [experts + 1] on the device, as ``moe.Plan.offsets``; None stands for one group of all the rows.
A group's values are whole numbers of -7 to 7 times a bfloat16 scale, the smallest that reaches a seventh of the group's
largest magnitude.  The products take x as it is (bfloat16, float16 or float32, any row stride), sum in float32 and round
once.  They are made for a few rows for each expert, where the weights' bytes count: from about sixteen rows for an expert on
``fp8.matmul`` is the faster one (16 experts of 2048 x 7168, one row each: 33 us against 48 with ``fp8.quantize``; eight 36
and 49, sixteen 49 and 49, 128 237 and 60).  Any number is right.  Every call runs on ``stream`` (default: the current one) and does not
synchronize.

Results have no autograd history, and these weights have no gradients: a tensor that requires one is refused while
gradients are recorded.
"""
from __future__ import annotations

import torch

from ._tensors import TYPES, native, on

GROUP = 128
ROWS = 16
RECORD = GROUP * ROWS // 2


class Matrix:
    """A matrix of n x k weights (or one for each expert) in 4 bits, in records of 16 rows x 128 columns.

    data     uint8 [tiles, blocks, 1024] or [experts, tiles, blocks, 1024], tiles = ceil(n / 16), blocks = ceil(k / 128)
    scales   bfloat16 [tiles, blocks, 16] or [experts, tiles, blocks, 16]: one for each row of a record

    Row r and column c of a record are in its 32-bit word ((r // 8) * 32 + (r % 8) * 4 + c // 32) * 4 + c % 32 // 8, from
    bit 4 * (c % 8 // 2 + 4 * (c % 2)) on, as the whole number + 8.
    """

    __slots__ = ("data", "scales", "rows", "cols")

    def __init__(self, data, scales, rows, cols):
        if data.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
            raise TypeError("data must be uint8 and scales bfloat16")
        if data.device != scales.device:
            raise ValueError(f"data is on {data.device}, scales on {scales.device}")
        if not (data.is_contiguous() and scales.is_contiguous()):
            raise ValueError("data and scales must be contiguous")
        shape = data.shape
        if rows < 1 or cols < 1 or len(shape) not in (3, 4) or shape[-3:] != (-(-rows // ROWS), -(-cols // GROUP), RECORD):
            raise ValueError(f"{rows} x {cols} weights cannot have records of the shape {tuple(shape)}")
        if scales.shape != (*shape[:-1], ROWS):
            raise ValueError(f"records of {tuple(shape)} cannot have scales of the shape {tuple(scales.shape)}")
        self.data, self.scales, self.rows, self.cols = data, scales, rows, cols

    def values(self, dtype=torch.float32, stream=None) -> torch.Tensor:
        """The weights that it stands for, [n, k] or [experts, n, k], each rounded once to `dtype`."""
        return on(stream, (self.data, self.scales), native.values4, self.data, self.scales, self.rows, self.cols, _type(dtype))


def _type(dtype):
    t = TYPES.get(dtype)
    if t is None:
        raise TypeError(f"the type must be bfloat16, float16 or float32, got {dtype}")
    return t


def _made(data, scales, rows, cols):
    """A Matrix of this module's own making: its parts fit and are not looked at again."""
    m = object.__new__(Matrix)
    m.data, m.scales, m.rows, m.cols = data, scales, rows, cols
    return m


def quantize_weight(w, stream=None) -> Matrix:
    """Weights [n, k] or [experts, n, k] (bfloat16, float16 or float32) in 4 bits; a group that holds an infinity or a NaN
    becomes NaN."""
    data, scales = on(stream, (w,), native.quantize4, w)
    return _made(data, scales, *w.shape[-2:])


def matmul(x, w: Matrix, offsets=None, out_dtype=None, stream=None) -> torch.Tensor:
    """x [rows, k] times the transpose of its group's w [n, k]: [rows, n] of ``out_dtype`` (default: x's), zeros for rows
    behind the last group.

    w holds one matrix for each group (data [groups, tiles, blocks, 1024]), or a single one without offsets."""
    if not isinstance(w, Matrix):
        raise TypeError("w must be a Matrix")
    return on(stream, (x, w.data, w.scales, offsets), native.matmul4, x, w.data, w.scales, w.rows, w.cols, offsets,
              None if out_dtype is None else _type(out_dtype))
