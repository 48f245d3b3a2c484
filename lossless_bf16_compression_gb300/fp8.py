"""8-bit floating point in blocks of 128 with a power-of-two scale each, and the experts' products on it.

    w, w_t = quantize_weight(weight)                      # [experts, n, k] -> blocks of 128 x 128, and the transpose
    y = matmul(quantize(x), w, offsets)                   # rows offsets[e] .. offsets[e + 1] - 1 times expert e's w^T
    dx = matmul(quantize(dy), w_t, offsets)
    dw = weight_grad(quantize_columns(dy, offsets), quantize_columns(x, offsets))   # [experts, n, k]

``offsets`` is int32 [experts + 1] on the device, as ``moe.Plan.offsets``; None stands for one group of all the rows.
A scale is the smallest power of two that brings its block's largest finite magnitude into the format's range, so
scaling is exact and only the rounding to 8 bits loses anything.  Sums are taken in float32.  Every call runs on
``stream`` (default: the current one) and does not synchronize.

Results have no autograd history: the gradients are the calls above.  A tensor that requires a gradient is refused while
gradients are recorded; use these calls under ``torch.no_grad``, on detached tensors or in a ``torch.autograd.Function``.
"""
from __future__ import annotations

import torch

from ._tensors import TYPES, native, on

BLOCK = 128
FORMATS = {"e4m3": 0, "e5m2": 1}


class Matrix:
    """A matrix (or one for each expert) in 8-bit blocks.

    data     uint8 [rows, pitch] or [experts, rows, pitch], pitch = 128 ceil(cols / 128); zeros past cols
    scales   uint8 [words, rows, 4] or [experts, words, rows, 4], words = ceil(pitch / 512): the scale of row r and
             block b is 2^(scales[..., b // 4, r, b % 4] - 127)
    cols     values in a row
    fmt      "e4m3" or "e5m2"
    offsets  from quantize_columns: the first block of each group, int32 [groups + 1]
    """

    __slots__ = ("data", "scales", "cols", "fmt", "offsets")

    def __init__(self, data, scales, cols, fmt="e4m3", offsets=None):
        _format(fmt)
        if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("data and scales must be uint8")
        if data.device != scales.device:
            raise ValueError(f"data is on {data.device}, scales on {scales.device}")
        if offsets is not None and not (isinstance(offsets, torch.Tensor) and offsets.dtype == torch.int32):
            raise TypeError("offsets must be an int32 tensor")
        if not (data.is_contiguous() and scales.is_contiguous()):
            raise ValueError("data and scales must be contiguous")
        shape, pitch = data.shape, _pitch(cols)
        if len(shape) not in (2, 3) or cols < 0 or shape[-1] != pitch:
            raise ValueError(f"rows of {cols} values take {pitch} bytes, data is {tuple(shape)}")
        if scales.shape != (*shape[:-2], -(-pitch // 512), shape[-2], 4):
            raise ValueError(f"scales of {tuple(shape)} cannot have the shape {tuple(scales.shape)}")
        self.data, self.scales, self.cols, self.fmt, self.offsets = data, scales, cols, fmt, offsets

    @property
    def rows(self) -> int:
        return self.data.shape[-2]

    def values(self) -> torch.Tensor:
        """The 8-bit values without their scales (a view)."""
        return native.values(self.data, FORMATS[self.fmt], self.cols)

    def scale_values(self, stream=None) -> torch.Tensor:
        """The scales as float32 powers of two, in their own layout."""
        return on(stream, (self.scales,), native.scale_values, self.scales)


def _made(data, scales, cols, fmt, offsets=None):
    """A Matrix of this module's own making: its parts fit and are not looked at again."""
    m = object.__new__(Matrix)
    m.data, m.scales, m.cols, m.fmt, m.offsets = data, scales, cols, fmt, offsets
    return m


def _pitch(cols):
    return -(-cols // BLOCK) * BLOCK


def _format(fmt):
    f = FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"fmt must be one of {', '.join(FORMATS)}, got {fmt!r}")
    return f


def quantize(x, fmt: str = "e4m3", stream=None) -> Matrix:
    """x [rows, cols] (bfloat16, float16 or float32, any row stride) in blocks of 128 along its rows."""
    data, scales = on(stream, (x,), native.quantize, x, _format(fmt))
    return _made(data, scales, x.shape[1], fmt)


def quantize_columns(x, offsets=None, fmt: str = "e4m3", stream=None) -> Matrix:
    """The transpose of x [rows, cols] in blocks of 128 of each group's rows, each group starting a block of its own.

    The result has `cols` rows; its ``offsets`` hold the first block of each group.  Blocks behind the last group's
    are zeros."""
    data, scales, starts = on(stream, (x, offsets), native.quantize_columns, x, offsets, _format(fmt))
    return _made(data, scales, data.shape[1], fmt, starts)


def quantize_weight(w, fmt: str = "e4m3", transposed: bool = True, stream=None) -> tuple[Matrix, Matrix | None]:
    """Weights [n, k] or [experts, n, k] in blocks of 128 x 128, and (with `transposed`) the same values transposed."""
    data, scales, data_t, scales_t = on(stream, (w,), native.quantize_weight, w, _format(fmt), bool(transposed))
    n, k = w.shape[-2:]
    return _made(data, scales, k, fmt), _made(data_t, scales_t, n, fmt) if transposed else None


def _product(stream, f, names, a, b, offsets, out_dtype):
    for name, m in zip(names, (a, b)):
        if not isinstance(m, Matrix):
            raise TypeError(f"{name} must be a Matrix")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return on(stream, (a.data, a.scales, b.data, b.scales, offsets), f, a.data, a.scales, FORMATS[a.fmt], a.cols,
              b.data, b.scales, FORMATS[b.fmt], b.cols, offsets, TYPES[out_dtype])


def matmul(a: Matrix, b: Matrix, offsets=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """a [rows, k] times the transpose of its group's b [n, k]: [rows, n], zeros for rows behind the last group.

    b holds one matrix for each group (data [groups, n, pitch]), or a single one without offsets."""
    return _product(stream, native.matmul, ("a", "b"), a, b, offsets, out_dtype)


def weight_grad(dy: Matrix, x: Matrix, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The gradient of matmul's weights, [groups, n, k], from quantize_columns of dy [rows, n] and x [rows, k]
    (with the same offsets); zeros for a group without rows."""
    both = isinstance(dy, Matrix) and isinstance(x, Matrix)
    if both and (dy.offsets is None or x.offsets is None):
        raise ValueError("dy and x must come from quantize_columns")
    if both and dy.offsets.shape != x.offsets.shape:
        raise ValueError("dy and x must have the same groups")
    return _product(stream, native.weight_grad, ("dy", "x"), dy, x, x.offsets if both else None, out_dtype)
