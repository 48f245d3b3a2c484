"""Plain 64-bit statements of the exchange and 8-bit block operators, on the CPU, for the tests.

They are written value by value from the definitions in include/zc_moe.h and share no code with the library.
"""
import numpy as np
import torch

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LEAST = {"e4m3": -6, "e5m2": -14}  # exponent of the smallest normal value


def sort(ids, experts):
    """(position [tokens, k], offsets [experts + 1]) of a routing (numpy int array [tokens, k])."""
    key = [int(v) if 0 <= int(v) < experts else experts for v in ids.reshape(-1)]
    order = sorted(range(len(key)), key=lambda s: (key[s], s))
    position = np.empty(len(key), dtype=np.int32)
    for place, s in enumerate(order):
        position[s] = place
    offsets = np.array([sum(k < e for k in key) for e in range(experts + 1)], dtype=np.int32)
    return position.reshape(ids.shape), offsets


def grid_values(fmt):
    """Every finite nonnegative value of the format, ascending."""
    m = MANTISSA[fmt]
    out = [i * 2.0 ** (LEAST[fmt] - m) for i in range(2 ** m)]
    e = LEAST[fmt]
    while out[-1] < TOP[fmt]:
        out += [v for v in ((1 + i / 2 ** m) * 2.0 ** e for i in range(2 ** m)) if v <= TOP[fmt]]
        e += 1
    return np.array(out)


def round_to_grid(v, fmt):
    """|v| <= TOP doubles to the nearest grid value, ties to the even mantissa (an even index in the grid)."""
    g = grid_values(fmt)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(g, a, side="left"), 0, len(g) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = g[hi] - a, a - g[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.copysign(np.where(take_hi, g[hi], g[lo]), v)


def block_scale(values, fmt):
    """The exponent of a block (1-D doubles, NaN and Inf allowed)."""
    finite = np.abs(values[np.isfinite(values)])
    amax = finite.max() if finite.size else 0.0
    if amax == 0:
        return 0
    s = -400
    while amax > TOP[fmt] * 2.0 ** s:
        s += 1
    return min(127, max(-127, s))


def quantize_blocks(x, fmt):
    """(values, exponents) of [rows, blocks, 128] doubles; an infinity is NaN where the format has none."""
    s = np.array([[block_scale(b, fmt) for b in row] for row in x]).reshape(x.shape[:2])
    v = x / 2.0 ** s[..., None].astype(np.float64)
    bad = ~np.isfinite(v)
    out = round_to_grid(np.where(bad, 0.0, v), fmt)
    odd = np.where(np.isinf(v), v if fmt == "e5m2" else np.nan, np.nan)
    return np.where(bad, odd, out), s


def quantize(x, fmt):
    """(values [rows, cols], exponents [rows, blocks]) of a [rows, cols] array."""
    r, c = x.shape
    wide = np.zeros((r, -(-c // 128) * 128))
    wide[:, :c] = x
    v, s = quantize_blocks(wide.reshape(r, -1, 128), fmt)
    return v.reshape(r, -1)[:, :c], s


def quantize_columns(x, offsets, fmt):
    """(values [cols, 128 capacity], exponents [cols, capacity], block offsets)."""
    rows, cols = x.shape
    groups = len(offsets) - 1
    capacity = rows // 128 + min(rows, groups)
    wide = np.zeros((cols, capacity * 128))
    starts, b = [], 0
    for g in range(groups):
        starts.append(b)
        a, z = offsets[g], offsets[g + 1]
        wide[:, b * 128:b * 128 + z - a] = x[a:z].T
        b += -(-(z - a) // 128)
    starts.append(b)
    v, s = quantize_blocks(wide.reshape(cols, capacity, 128), fmt)
    return v.reshape(cols, -1), s, np.array(starts, dtype=np.int32)


def unpack_scales(scales, blocks):
    """uint8 scales [..., words, rows, 4] as exponents [..., rows, blocks]."""
    s = np.asarray(scales).astype(np.int64) - 127
    s = np.moveaxis(s, -3, -2)
    return s.reshape(*s.shape[:-2], -1)[..., :blocks]


def dequantize(m):
    """The values that an fp8.Matrix stands for, as doubles [..., rows, cols] (padding cut)."""
    v = m.values().float().cpu().numpy().astype(np.float64)
    blocks = m.data.shape[-1] // 128
    s = unpack_scales(m.scales.cpu().numpy(), blocks)
    return v * np.repeat(2.0 ** s.astype(np.float64), 128, axis=-1)[..., : v.shape[-1]]


def doubles(t):
    return t.detach().double().cpu().numpy()


def half_ulp(dtype):
    """Largest relative error of one rounding to the type (normal values): 2^-p, p its significant bits."""
    return {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]


def smallest(dtype):
    """Half of the type's smallest positive value: the error of a rounding below the normal range."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[dtype]
