"""8-bit floating point in blocks of 128 with a power-of-two scale each, and the experts' products on it.

    w, w_t = quantize_weight(weight)                      # [experts, n, k] -> blocks of 128 x 128, and the transpose
    y = matmul(quantize(x), w, offsets)                   # rows offsets[e] .. offsets[e + 1] - 1 times expert e's w^T
    dx = matmul(quantize(dy), w_t, offsets)
    dw = weight_grad(quantize_columns(dy, offsets), quantize_columns(x, offsets))   # [experts, n, k]

``offsets`` is int32 [experts + 1] on the device, as ``moe.Plan.offsets``; None stands for one group of all the rows.
A scale is the smallest power of two that brings its block's largest finite magnitude into the format's range, so
scaling is exact and only the rounding to 8 bits loses anything.  Sums are taken in float32.  Every call runs on
``stream`` (default: the current one) and does not synchronize.
"""
from __future__ import annotations

import torch

from ._tensors import MAX_EXPERTS, TYPES, call, check, current, fn, on, on_device, rows_of

BLOCK = 128
FORMATS = {"e4m3": 0, "e5m2": 1}
_FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


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
        return self.data.view(_FLOAT8[self.fmt]).narrow(-1, 0, self.cols)

    def scale_values(self, stream=None) -> torch.Tensor:
        """The scales as float32 powers of two, in their own layout."""
        device = on_device("scales", self.scales, None)
        return on(stream, (self.scales,), _scale_values, self.scales, device)


_ROW_TYPES = tuple(TYPES)
_INT32 = (torch.int32,)


def _made(data, scales, cols, fmt, offsets=None):
    """A Matrix of this module's own making: its parts fit and are not looked at again."""
    m = object.__new__(Matrix)
    m.data, m.scales, m.cols, m.fmt, m.offsets = data, scales, cols, fmt, offsets
    return m


def _scale_values(scales, device):
    out = torch.empty(scales.shape, dtype=torch.float32, device=scales.device)
    call("zc_fp8_scale_values", scales.data_ptr(), scales.numel() // 4, out.data_ptr(), current(device))
    return out


def _pitch(cols):
    return -(-cols // BLOCK) * BLOCK


def _empty(lead, rows, cols, device):
    pitch = _pitch(cols)
    return (torch.empty((*lead, rows, pitch), dtype=torch.uint8, device=device),
            torch.empty((*lead, -(-pitch // 512), rows, 4), dtype=torch.uint8, device=device))


def _format(fmt):
    f = FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"fmt must be one of {', '.join(FORMATS)}, got {fmt!r}")
    return f


def _input(name, x):
    device = on_device(name, x, None, _ROW_TYPES, 2)
    if x.shape[1] < 1:
        raise ValueError(f"{name} must have at least one column")
    return device


def _offsets(offsets, device):
    if offsets is None:
        return 1, None
    on_device("offsets", offsets, device, _INT32, 1)
    if not 2 <= offsets.shape[0] <= MAX_EXPERTS + 1:
        raise ValueError(f"offsets must have 2 to {MAX_EXPERTS + 1} entries")
    if not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous")
    return offsets.shape[0] - 1, offsets.data_ptr()


def quantize(x, fmt: str = "e4m3", stream=None) -> Matrix:
    """x [rows, cols] (bfloat16, float16 or float32, any row stride) in blocks of 128 along its rows."""
    f = _format(fmt)
    device = _input("x", x)
    return on(stream, (x,), _quantize, x, f, fmt, device)


def _quantize(x, f, fmt, device):
    x, pitch = rows_of(x)
    rows, cols = x.shape
    data, scales = _empty((), rows, cols, x.device)
    call("zc_fp8_quantize", x.data_ptr(), pitch, TYPES[x.dtype], rows, cols, f, data.data_ptr(), scales.data_ptr(),
         current(device))
    return _made(data, scales, cols, fmt)


def quantize_columns(x, offsets=None, fmt: str = "e4m3", stream=None) -> Matrix:
    """The transpose of x [rows, cols] in blocks of 128 of each group's rows, each group starting a block of its own.

    The result has `cols` rows; its ``offsets`` hold the first block of each group.  Blocks behind the last group's
    are zeros."""
    f = _format(fmt)
    device = _input("x", x)
    groups, at = _offsets(offsets, device)
    return on(stream, (x, offsets), _quantize_columns, x, groups, at, f, fmt, device)


def _quantize_columns(x, groups, at, f, fmt, device):
    x, pitch = rows_of(x)
    rows, cols = x.shape
    wide = fn("zc_fp8_column_blocks")(rows, groups) * BLOCK
    data, scales = _empty((), cols, wide, x.device)
    starts = torch.empty(groups + 1, dtype=torch.int32, device=x.device)
    call("zc_fp8_quantize_columns", x.data_ptr(), pitch, TYPES[x.dtype], rows, cols, groups, at, f, data.data_ptr(),
         scales.data_ptr(), starts.data_ptr(), current(device))
    return _made(data, scales, wide, fmt, starts)


def quantize_weight(w, fmt: str = "e4m3", transposed: bool = True, stream=None) -> tuple[Matrix, Matrix | None]:
    """Weights [n, k] or [experts, n, k] in blocks of 128 x 128, and (with `transposed`) the same values transposed."""
    f = _format(fmt)
    device = on_device("w", w, None, _ROW_TYPES)
    check(w.dim() in (2, 3) and min(w.shape) >= 1, f"w must be [n, k] or [experts, n, k], got {tuple(w.shape)}")
    check(w.dim() == 2 or w.shape[0] <= MAX_EXPERTS, f"at most {MAX_EXPERTS} experts")
    return on(stream, (w,), _quantize_weight, w, f, fmt, transposed, device)


def _quantize_weight(w, f, fmt, transposed, device):
    w = w.contiguous()
    lead, n, k = tuple(w.shape[:-2]), *w.shape[-2:]
    data, scales = _empty(lead, n, k, w.device)
    data_t, scales_t = _empty(lead, k, n, w.device) if transposed else (None, None)
    call("zc_fp8_quantize_weight", w.data_ptr(), TYPES[w.dtype], lead[0] if lead else 1, n, k, f, data.data_ptr(),
         scales.data_ptr(), data_t.data_ptr() if transposed else None, scales_t.data_ptr() if transposed else None,
         current(device))
    return _made(data, scales, k, fmt), _made(data_t, scales_t, n, fmt) if transposed else None


def _out_type(dtype):
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {dtype}")
    return TYPES[dtype]


def _operand(name, m, device, dim=None):
    if not isinstance(m, Matrix):
        raise TypeError(f"{name} must be a Matrix")
    return on_device(name, m.data, device, None, dim)


def matmul(a: Matrix, b: Matrix, offsets=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """a [rows, k] times the transpose of its group's b [n, k]: [rows, n], zeros for rows behind the last group.

    b holds one matrix for each group (data [groups, n, pitch]), or a single one without offsets."""
    t = _out_type(out_dtype)
    device = _operand("a", a, None, 2)
    _operand("b", b, device)
    groups, at = _offsets(offsets, device)
    if a.cols != b.cols or a.cols < 1:
        raise ValueError(f"a has rows of {a.cols} values, b of {b.cols}")
    held = b.data.shape
    if (held[0] if len(held) == 3 else 1) != groups:
        raise ValueError(f"b must hold {groups} matrices, got {tuple(held)}")
    return on(stream, (a.data, a.scales, b.data, b.scales, offsets), _matmul, a, b, groups, at, out_dtype, t, device)


def _matmul(a, b, groups, at, out_dtype, t, device):
    a_data, b_data, k = a.data, b.data, a.cols
    rows, n = a_data.shape[0], b_data.shape[-2]
    out = torch.empty((rows, n), dtype=out_dtype, device=a_data.device)
    need = fn("zc_fp8_matmul_workspace")(rows, groups, n, k)
    scratch = torch.empty(need, dtype=torch.uint8, device=a_data.device) if need else None
    call("zc_fp8_matmul", a_data.data_ptr(), a.scales.data_ptr(), FORMATS[a.fmt], rows, b_data.data_ptr(),
         b.scales.data_ptr(), FORMATS[b.fmt], groups, n, k, at, out.data_ptr(), n, t,
         None if scratch is None else scratch.data_ptr(), current(device))
    return out


def weight_grad(dy: Matrix, x: Matrix, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The gradient of matmul's weights, [groups, n, k], from quantize_columns of dy [rows, n] and x [rows, k]
    (with the same offsets); zeros for a group without rows."""
    t = _out_type(out_dtype)
    device = _operand("dy", dy, None, 2)
    _operand("x", x, device, 2)
    check(dy.offsets is not None and x.offsets is not None, "dy and x must come from quantize_columns")
    check(dy.cols == x.cols and dy.offsets.shape == x.offsets.shape, "dy and x must have the same groups")
    groups, at = _offsets(x.offsets, device)
    return on(stream, (dy.data, dy.scales, x.data, x.scales, x.offsets), _weight_grad, dy, x, groups, at, out_dtype, t,
              device)


def _weight_grad(dy, x, groups, at, out_dtype, t, device):
    out = torch.empty((groups, dy.rows, x.rows), dtype=out_dtype, device=x.data.device)
    call("zc_fp8_weight_grad", dy.data.data_ptr(), dy.scales.data_ptr(), FORMATS[dy.fmt], x.data.data_ptr(),
         x.scales.data_ptr(), FORMATS[x.fmt], x.cols // BLOCK, groups, dy.rows, x.rows, at, out.data_ptr(), t,
         current(device))
    return out
