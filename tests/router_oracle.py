"""Plain 64-bit statements of a router's operators and of 4-bit weights, on the CPU, for the tests.

They are written row by row from the definitions in include/zc_router.h and include/zc_int4.h and share no code with the
library.
"""
import numpy as np


# ------------------------------------------------------------------ the router


def choose(logits, k):
    """Experts of each row's k largest logits: NaN above all, equal ones by index, -1 where only -infinity is left."""
    out = np.full((len(logits), k), -1, dtype=np.int32)
    for t, row in enumerate(logits):
        order = sorted(range(len(row)), key=lambda e: (0 if np.isnan(row[e]) else 1, 0.0 if np.isnan(row[e]) else -row[e], e))
        order = [e for e in order if not row[e] == -np.inf][:k]
        out[t, : len(order)] = order
    return out


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softmax(x):
    """Of a row; zeros for a row of nothing but -infinity."""
    if len(x) == 0 or (x == -np.inf).all():
        return np.zeros_like(x)
    with np.errstate(invalid="ignore"):
        top = np.nan if np.isnan(x).any() else x.max()
        e = np.exp(x - top)
    return e / e.sum()


def shares(x):
    """Sigmoids divided by their sum, by their logarithms, so that low ones do not vanish."""
    return softmax(-np.logaddexp(0, -x))


def weights(logits, ids, score, normalize, scale=1.0):
    out = np.zeros(ids.shape)
    for t, row in enumerate(logits):
        slots = np.flatnonzero((ids[t] >= 0) & (ids[t] < len(row)))
        x = row[ids[t][slots]]
        if score == "softmax":
            w = softmax(x) if normalize else softmax(row)[ids[t][slots]]
        else:
            w = shares(x) if normalize else sigmoid(x)
        out[t, slots] = scale * w
    return out


def route_grad(d_weights, logits, ids, score, normalize, scale=1.0):
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        slots = np.flatnonzero((ids[t] >= 0) & (ids[t] < len(row)))
        slots = slots[row[ids[t][slots]] != -np.inf]
        e, g = ids[t][slots], scale * d_weights[t][slots]
        x = row[e]
        if score == "softmax" and not normalize:
            p = softmax(row)
            out[t] = -p * (g * p[e]).sum()
            np.add.at(out[t], e, p[e] * g)
            continue
        if score == "softmax":
            w = softmax(x)
            d = w * (g - (g * w).sum())
        elif normalize:
            w = shares(x)
            d = w * (1 - sigmoid(x)) * (g - (g * w).sum())
        else:
            d = sigmoid(x) * (1 - sigmoid(x)) * g
        np.add.at(out[t], e, d)
    return out


def probabilities(logits, score):
    p = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        if not (row == -np.inf).all():
            p[t] = softmax(row) if score == "softmax" else shares(row)
    return p


def balance(logits, ids, score):
    """(loss, counts, slope)."""
    tokens, experts = logits.shape
    counts = np.array([(ids == e).sum() for e in range(experts)], dtype=np.int64)
    n = int((logits != -np.inf).any(1).sum())
    if n == 0:
        return 0.0, counts, np.zeros(experts)
    slope = experts * counts / (ids.shape[1] * float(n) * n)
    return float((slope * probabilities(logits, score).sum(0)).sum()), counts, slope


def balance_grad(d_loss, logits, slope, score):
    p = probabilities(logits, score)
    d = p * (slope - (p * slope).sum(1, keepdims=True)) * d_loss
    return d * (1 - sigmoid(logits)) if score == "sigmoid" else d


# ------------------------------------------------------------------ 4-bit weights


def bf16_at_least(v):
    """The smallest bfloat16 value (as a double) that is at least the double v > 0."""
    unit = 2.0 ** max(np.frexp(v)[1] - 8, -133)
    return np.ceil(v / unit) * unit


def quantize(w):
    """(q [n, blocks, 128], scales [n, blocks]) of doubles [n, k]; scale NaN and q = 0 where a group is not finite."""
    n, k = w.shape
    wide = np.zeros((n, -(-k // 128) * 128))
    wide[:, :k] = w
    wide = wide.reshape(n, -1, 128)
    q, scales = np.zeros(wide.shape, dtype=np.int64), np.ones(wide.shape[:2])
    for r in range(n):
        for b in range(wide.shape[1]):
            v = wide[r, b]
            if not np.isfinite(v).all():
                scales[r, b] = np.nan
                continue
            amax = np.abs(v).max()
            if amax == 0:
                continue
            s = bf16_at_least(amax / 7)
            while 7 * s < amax:  # (amax / 7 was rounded down to a bfloat16 value)
                s = bf16_at_least(s * (1 + 2.0 ** -20))
            scales[r, b] = s
            q[r, b] = np.rint(v / s)
    return q, scales


def unpack(data, scales, n, k):
    """(q [n, blocks, 128], scales [n, blocks]) of one matrix's records, word by word as the header numbers them."""
    tiles, blocks, _ = data.shape
    words = np.ascontiguousarray(data).view("<u4").reshape(tiles, blocks, 256)
    q = np.zeros((tiles * 16, blocks, 128), dtype=np.int64)
    for r in range(16):
        for c in range(128):
            word = words[:, :, ((r // 8) * 32 + (r % 8) * 4 + c // 32) * 4 + c % 32 // 8]
            q[r::16, :, c] = (word >> (4 * (c % 8 // 2 + 4 * (c % 2)))).astype(np.int64) % 16 - 8
    s = scales.transpose(0, 2, 1).reshape(tiles * 16, blocks)
    return q[:n], s[:n], q[n:], s[n:]


def pack(q, s):
    """Records uint8 [tiles, blocks, 1024] of q [n, blocks, 128], and scales [tiles, blocks, 16]."""
    n, blocks, _ = q.shape
    tiles = -(-n // 16)
    u = np.full((tiles * 16, blocks, 128), 8, dtype=np.uint32)
    u[:n] = q + 8
    words = np.zeros((tiles, blocks, 256), dtype="<u4")
    for r in range(16):
        for c in range(128):
            words[:, :, ((r // 8) * 32 + (r % 8) * 4 + c // 32) * 4 + c % 32 // 8] |= u[r::16, :, c] << (4 * (c % 8 // 2 + 4 * (c % 2)))
    scales = np.ones((tiles * 16, blocks))
    scales[:n] = s
    return words.view(np.uint8).reshape(tiles, blocks, 1024), scales.reshape(tiles, 16, blocks).transpose(0, 2, 1).copy()


def weight_values(q, s, k):
    return (q * s[..., None]).reshape(q.shape[0], -1)[:, :k]
