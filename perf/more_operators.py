"""Timed cases of the router of an expert layer (its choice of experts, its balance loss, their gradients) and of the
experts' products on 4-bit weights, for decoding.

Each case is one call (or one forward and backward step of a router) as a user's program makes it.  ``run`` computes it
in plain torch operations in 32 bits, or, with ``own`` set, through the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = 128  # weights along a row that share a scale
RECORD = 16 * GROUP // 2  # bytes of 16 rows x 128 weights


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a decode step: latency only
        dict(name="route_one_token", op="route", tokens=1, experts=64, k=8, dtype="fp32", score="softmax", normalize=True, masked=0.0, padded=0.0),
        # a ragged prompt whose tokens may use part of the experts, in 16 bits (equal logits happen), some rows padding
        dict(name="route_odd", op="route", tokens=4999, experts=40, k=6, dtype="fp16", score="sigmoid", normalize=False, masked=0.3, padded=0.1),
        # the backward step of the weights alone, many experts
        dict(name="route_grad_train", op="route_grad", tokens=16384, experts=256, k=8, dtype="fp32", score="sigmoid", normalize=True, masked=0.0, padded=0.0),
        # the balance loss of a small padded batch and its gradient
        dict(name="balance_odd", op="balance", tokens=777, experts=40, k=6, dtype="fp16", score="softmax", normalize=True, masked=0.0, padded=0.2),
        # the balance loss of a training step and its gradient
        dict(name="balance_train", op="balance", tokens=32768, experts=64, k=8, dtype="fp32", score="softmax", normalize=True, masked=0.0, padded=0.0),
        # a router's training step: choice, loss, and the gradient of both
        dict(name="router_step", op="router", tokens=16384, experts=256, k=8, dtype="bf16", score="softmax", normalize=True, masked=0.0, padded=0.0),
        # the weights of 16 experts made 4-bit, and their values
        dict(name="int4_quantize", op="quantize", experts=16, out=2048, cols=7168, dtype="bf16"),
        # one matrix of odd sizes
        dict(name="int4_quantize_odd", op="quantize", experts=1, out=777, cols=1000, dtype="fp32"),
        # one token and one matrix: a matrix-vector product
        dict(name="int4_one_row", op="matmul", rows=1, experts=1, out=4096, cols=7168, dtype="bf16"),
        # one token and its eight experts of 64
        dict(name="int4_one_token", op="matmul", rows=8, experts=64, out=2048, cols=7168, dtype="bf16"),
        # a decode batch of 64 tokens and eight experts each
        dict(name="int4_batch", op="matmul", rows=512, experts=64, out=2048, cols=7168, dtype="bf16"),
        # a few rows on small experts of odd sizes
        dict(name="int4_odd", op="matmul", rows=37, experts=8, out=1999, cols=1000, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "balance", "router", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("route", "route_grad", "balance", "router"):
        experts = _log(rng, 8, 256)
        normalize = rng.random() < 0.7
        return dict(op=op, tokens=_log(rng, 1, 32768 if experts <= 128 else 16384), experts=experts,
                    k=rng.randint(2 if normalize else 1, 8),  # a single normalized weight is 1, without a gradient
                    dtype=dtype, score=rng.choice(["softmax", "sigmoid"]), normalize=normalize,
                    masked=rng.choice([0.0, 0.0, 0.3]), padded=rng.choice([0.0, 0.0, 0.15]))
    experts, out, cols = _log(rng, 1, 64), _log(rng, 64, 4096), _log(rng, 64, 7168)
    if rng.random() < 0.6:
        out, cols = 16 * max(1, out // 16), 128 * max(1, cols // 128)
    most = 16 if op == "quantize" else 64
    while experts * out * cols > most * 2048 * 7168:
        experts //= 2
    if op == "quantize":
        return dict(op=op, experts=experts, out=out, cols=cols, dtype=dtype)
    return dict(op=op, rows=_log(rng, 1, 512), experts=experts, out=out, cols=cols, dtype=dtype)


def work(case):
    c, b = case, BYTES[case["dtype"]]
    if "tokens" in c:
        te, tk, e = c["tokens"] * c["experts"], c["tokens"] * c["k"], c["experts"]
        return {
            "route": {"bytes": te * b + 8 * tk, "flops": 4 * te},
            # the chosen logits, their experts and gradients in; a whole row out
            "route_grad": {"bytes": te * b + tk * (8 + b) + (0 if c["normalize"] or c["score"] == "sigmoid" else te * b), "flops": 8 * tk},
            "balance": {"bytes": 2 * te * b + 4 * tk + 8 * e + 4, "flops": 10 * te},
            "router": {"bytes": 2 * te * b + 12 * tk + 8 * e + 4, "flops": 14 * te},
        }[c["op"]]
    n, k, e = c["out"], c["cols"], c["experts"]
    if c["op"] == "quantize":
        return {"bytes": e * n * (2 * k * b + k // 2 + 2 * -(-k // GROUP)), "flops": 3 * e * n * k}
    active = e * (1.0 - (1.0 - 1.0 / e) ** c["rows"])  # experts that get a row, on average
    return {"bytes": int(active * n * (k / 2 + 2 * -(-k // GROUP)) + c["rows"] * (k + n) * b), "flops": 2 * c["rows"] * n * k}


# ------------------------------------------------------------------ inputs


def _logits(c, g):
    """A router's logits: some experts more popular than others; masked experts and padding rows are -infinity."""
    t, e = c["tokens"], c["experts"]
    x = torch.randn((t, e), generator=g, device=DEV) * 1.5 + torch.randn(e, generator=g, device=DEV) * 0.5
    if c["masked"]:
        x = torch.where(torch.rand((t, e), generator=g, device=DEV) < c["masked"], -math.inf, x)
    if c["padded"]:
        x = torch.where(torch.rand((t, 1), generator=g, device=DEV) < c["padded"], -math.inf, x)
    return x.to(DTYPES[c["dtype"]])


def _codes(w):
    """Rows of weights [n, k] as whole numbers -7 .. 7 and the scales of groups of 128 (a short last group as it is): a
    scale is the smallest bfloat16 value of at least a seventh of the group's largest magnitude, 1 for a group of zeros."""
    n, k = w.shape
    w = torch.nn.functional.pad(w.float(), (0, -k % GROUP)).view(n, -1, GROUP)
    amax = w.abs().amax(2)
    s = (((amax / 7.0).view(torch.int32) >> 16) << 16).view(torch.float32)
    s = torch.where(7.0 * s < amax, (s.view(torch.int32) + 0x10000).view(torch.float32), s)
    s = torch.where(amax > 0, s, 1.0)
    return w, s


def _pack(q, s):
    """Whole numbers [n, blocks, 128] and scales [n, blocks] in the library's layout: for each 16 rows and group of 128 a
    record of 1024 bytes (values + 8; 8 rows x 4 parts of 32 weights x 4 words, twice), and 16 bfloat16 scales."""
    n, blocks, _ = q.shape
    tiles = -(-n // 16)
    u = torch.full((tiles * 16, blocks, GROUP), 8, dtype=torch.uint8, device=q.device)
    u[:n] = (q + 8).to(torch.uint8)
    u = u.view(tiles, 2, 8, blocks, 4, 4, 8).permute(0, 3, 1, 2, 4, 5, 6)
    data = u[..., [0, 4, 1, 5]] | (u[..., [2, 6, 3, 7]] << 4)
    scales = torch.ones((tiles * 16, blocks), dtype=torch.bfloat16, device=q.device)
    scales[:n] = s.to(torch.bfloat16)
    return data.reshape(tiles, blocks, RECORD), scales.view(tiles, 16, blocks).permute(0, 2, 1).contiguous()


def _groups(c, seed):
    """Rows of each expert, on the host: a skewed choice for each row."""
    rng = np.random.default_rng(seed)
    p = np.exp(0.3 * rng.standard_normal(c["experts"]))
    counts = rng.multinomial(c["rows"], p / p.sum())
    return [0] + [int(v) for v in np.cumsum(counts)]


def _inputs(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(seed)
    d = DTYPES[c["dtype"]]
    s = {"case": dict(c)}
    if "tokens" in c:
        s["logits"] = _logits(c, g)
        if c["op"] != "route":
            scale = 4096.0 if c["dtype"] == "fp16" else 1.0  # as training in fp16 scales its loss
            s["d_weights"] = torch.randn((c["tokens"], c["k"]), generator=g, device=DEV) * (1e-3 * scale)
            s["d_loss"] = torch.full((), 0.01 * scale, device=DEV)
        if c["op"] in ("route_grad", "balance"):
            s["ids"] = _choose(s["logits"], c["k"])[1]  # what the forward step chose
        return s
    e, n, k = c["experts"], c["out"], c["cols"]
    if c["op"] == "quantize":
        s["w"] = (torch.randn((e, n, k), generator=g, device=DEV) * 0.02).to(d)
        return s
    # the weights as a program loads them
    s["data"] = torch.empty((e, -(-n // 16), -(-k // GROUP), RECORD), dtype=torch.uint8, device=DEV)
    s["scales"] = torch.empty((e, -(-n // 16), -(-k // GROUP), 16), dtype=torch.bfloat16, device=DEV)
    for i in range(e):
        w, scale = _codes(torch.randn((n, k), generator=g, device=DEV) * 0.02)
        s["data"][i], s["scales"][i] = _pack(torch.round(w / scale[..., None]), scale)
    s["host_offsets"] = _groups(c, seed)
    s["offsets"] = torch.tensor(s["host_offsets"], dtype=torch.int32, device=DEV) if e > 1 else None
    x = torch.randn((c["rows"], k), generator=g, device=DEV)
    s["x"] = (x * torch.where(torch.rand(k, generator=g, device=DEV) < 0.002, 20.0, 1.0)).to(d)  # a few loud channels
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ------------------------------------------------------------------ the plain forms


def _choose(logits, k):
    """The k largest logits of each row and their experts, equal ones by index; no expert (-1) where only -infinity is left."""
    top, ids = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    return top, torch.where(top > -math.inf, ids, -1).to(torch.int32)


def _scores(x, score):
    """A row's softmax, or sigmoids; 0 in rows of nothing but -infinity."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    return p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _route(logits, c):
    x = logits.float()
    top, ids = _choose(logits, c["k"])
    if c["score"] == "softmax" and not c["normalize"]:
        s = torch.gather(_scores(x, "softmax"), 1, ids.long().clamp(min=0))
    else:
        s = _scores(top, c["score"])
    s = torch.where(ids >= 0, s, 0.0)
    if c["normalize"] and c["score"] == "sigmoid":
        s = s / s.sum(1, keepdim=True).clamp(min=1e-30)
    return s, ids


def _route_grad(d_weights, logits, ids, c):
    """The gradient of the weights with respect to the logits, in 32 bits."""
    x, at = logits.float(), ids.long().clamp(min=0)
    kept = ids >= 0
    g = torch.where(kept, d_weights, 0.0)
    top = torch.where(kept, torch.gather(x, 1, at), -math.inf)
    if c["score"] == "softmax" and not c["normalize"]:
        p = _scores(x, "softmax")
        full = torch.zeros_like(x).scatter_add_(1, at, g)
        return p * (full - (full * p).sum(1, keepdim=True))
    s = _scores(top, c["score"])
    if c["score"] == "softmax":
        d = s * (g - (g * s).sum(1, keepdim=True))
    elif c["normalize"]:
        w = s / s.sum(1, keepdim=True).clamp(min=1e-30)
        d = w * (1.0 - s) * (g - (g * w).sum(1, keepdim=True))
    else:
        d = s * (1.0 - s) * g
    return torch.zeros_like(x).scatter_add_(1, at, torch.where(kept, d, 0.0))


def _probabilities(logits, score):
    x = logits.float()
    if score == "softmax":
        return _scores(x, "softmax"), 1.0
    s = _scores(x, "sigmoid")
    return s / s.sum(1, keepdim=True).clamp(min=1e-30), 1.0 - s


def _balance(logits, ids, c):
    """Loss, counts and the loss's slope in each expert's probability."""
    e = c["experts"]
    p, _ = _probabilities(logits, c["score"])
    n = (logits > -math.inf).any(1).sum().double()
    counts = (ids.reshape(-1)[:, None] == torch.arange(e, device=ids.device, dtype=torch.int32)).sum(0)
    slope = torch.where(n > 0, e * counts.double() / (c["k"] * n * n).clamp(min=1.0), 0.0)
    loss = (slope * p.sum(0, dtype=torch.float64)).sum()
    return loss.float(), counts.to(torch.int32), slope.float()


def _balance_grad(d_loss, logits, slope, c):
    p, rest = _probabilities(logits, c["score"])
    return d_loss * p * rest * (slope - (slope * p).sum(1, keepdim=True))


def _weight(data, scales, n, k):
    """One matrix in 4 bits as its 32-bit values [n, k]."""
    tiles, blocks, _ = data.shape
    b = data.view(tiles, blocks, 2, 8, 4, 4, 4)
    q = torch.stack([b[..., 0] & 15, b[..., 2] & 15, b[..., 0] >> 4, b[..., 2] >> 4,
                     b[..., 1] & 15, b[..., 3] & 15, b[..., 1] >> 4, b[..., 3] >> 4], -1).float() - 8.0
    q = q.permute(0, 2, 3, 1, 4, 5, 6).reshape(tiles * 16, blocks, GROUP)
    q = q * scales.float().permute(0, 2, 1).reshape(tiles * 16, blocks)[..., None]
    return q.view(tiles * 16, blocks * GROUP)[:n, :k]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _route(s["logits"], c)
    if op == "route_grad":
        return _route_grad(s["d_weights"], s["logits"], s["ids"], c).to(s["logits"].dtype)
    if op == "balance":
        loss, counts, slope = _balance(s["logits"], s["ids"], c)
        return loss, counts, slope, _balance_grad(s["d_loss"], s["logits"], slope, c).to(s["logits"].dtype)
    if op == "router":
        weights, ids = _route(s["logits"], c)
        loss, counts, slope = _balance(s["logits"], ids, c)
        d = _route_grad(s["d_weights"], s["logits"], ids, c) + _balance_grad(s["d_loss"], s["logits"], slope, c)
        return weights, ids, loss, counts, d.to(s["logits"].dtype)
    if op == "quantize":
        out = torch.empty_like(s["w"])
        for i in range(c["experts"]):
            w, scale = _codes(s["w"][i])
            wide = torch.float64 if c["dtype"] == "fp32" else torch.float32  # 24 bits may lie next to a half
            q = torch.round(w.to(wide) / scale[..., None].to(wide)).float() * scale[..., None]
            out[i] = q.view(c["out"], -1)[:, : c["cols"]].to(out.dtype)
        return out
    y = torch.zeros((c["rows"], c["out"]), device=s["x"].device)
    at = s["host_offsets"]
    for i in range(c["experts"]):
        if at[i] < at[i + 1]:
            y[at[i] : at[i + 1]] = s["x"][at[i] : at[i + 1]].float() @ _weight(s["data"][i], s["scales"][i], c["out"], c["cols"]).t()
    return y.to(s["x"].dtype)


# ------------------------------------------------------------------ the library's calls


def _own(s):
    from lossless_bf16_compression_gb300 import int4, moe

    c = s["case"]
    op = c["op"]
    if op == "route":
        return moe.route(s["logits"], c["k"], c["score"], c["normalize"])
    if op == "route_grad":
        return moe.route_grad(s["d_weights"], s["logits"], s["ids"], c["score"], c["normalize"])
    if op == "balance":
        b = moe.balance(s["logits"], s["ids"], c["score"])
        return b.loss, b.counts, b.slope, moe.balance_grad(s["d_loss"], s["logits"], b, c["score"])
    if op == "router":
        weights, ids = moe.route(s["logits"], c["k"], c["score"], c["normalize"])
        b = moe.balance(s["logits"], ids, c["score"])
        d = moe.route_grad(s["d_weights"], s["logits"], ids, c["score"], c["normalize"], balance=(s["d_loss"], b))
        return weights, ids, b.loss, b.counts, d
    if op == "quantize":
        return int4.quantize_weight(s["w"]).values(s["w"].dtype)
    w = int4.Matrix(s["data"], s["scales"], c["out"], c["cols"])
    return int4.matmul(s["x"], w, s["offsets"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits


def _weights64(logits, ids, c):
    """The weights of chosen experts, from the definition, differentiable."""
    kept = ids >= 0
    at = ids.long().clamp(min=0)
    if c["score"] == "softmax":
        dead = ~torch.isfinite(logits).any(1, keepdim=True)
        s = torch.softmax(torch.where(dead, 0.0, logits), 1).gather(1, at)
    else:
        s = torch.sigmoid(logits.gather(1, at))
    s = torch.where(kept, s, 0.0)
    if c["normalize"]:
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total > 0, total, 1.0)
    return s


def _ids64(logits, k):
    """Take the largest one k times, the lowest index among equals."""
    left, out = logits.clone(), []
    index = torch.arange(logits.shape[1], device=logits.device)
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        i = torch.where(left == top, index, logits.shape[1]).amin(1, keepdim=True)
        out.append(torch.where(top > -math.inf, i, -1))
        left = left.scatter(1, i, -math.inf)
    return torch.cat(out, 1)


def _loss64(logits, ids, c):
    dead = ~torch.isfinite(logits).any(1, keepdim=True)
    x = torch.where(dead, 0.0, logits)
    if c["score"] == "softmax":
        p = torch.softmax(x, 1)
    else:
        p = torch.sigmoid(x)
        p = p / p.sum(1, keepdim=True)
    p = torch.where(dead, 0.0, p)
    n = int((~dead).sum())
    counts = torch.bincount(ids[ids >= 0].long().reshape(-1), minlength=c["experts"]).double()
    if n == 0:
        return (p * 0.0).sum(), counts, counts * 0.0
    share = counts / (c["k"] * n)
    return c["experts"] * (share * p.sum(0) / n).sum(), counts, c["experts"] * share / n


def exact(case, seed):
    s, c = _inputs(case, seed), case
    op = c["op"]
    if "tokens" in c:
        logits = s["logits"].double().requires_grad_()
        ids = s["ids"] if "ids" in s else _ids64(logits.detach(), c["k"]) if c["k"] <= c["experts"] else None
        if op == "route":
            return _weights64(logits, ids, c).detach(), ids
        if op == "route_grad":
            return torch.autograd.grad((_weights64(logits, ids, c) * s["d_weights"].double()).sum(), logits)[0]
        loss, counts, slope = _loss64(logits, ids, c)
        total = loss * s["d_loss"].double()
        if op == "balance":
            return loss.detach(), counts, slope, torch.autograd.grad(total, logits)[0]
        weights = _weights64(logits, ids, c)
        d = torch.autograd.grad(total + (weights * s["d_weights"].double()).sum(), logits)[0]
        return weights.detach(), ids, loss.detach(), counts, d
    n, k = c["out"], c["cols"]
    if op == "quantize":
        out = torch.empty((c["experts"], n, k), dtype=torch.float64, device=DEV)
        for i in range(c["experts"]):
            for a in range(0, k, GROUP):
                w = s["w"][i, :, a : a + GROUP].double()
                amax = w.abs().amax(1, keepdim=True)
                m, e = torch.frexp(amax / 7.0)
                step = torch.ldexp(torch.ceil(m * 256.0) / 256.0, e)
                step = torch.where(7.0 * step < amax, step * (1.0 + 2.0 ** -7), step)
                step = torch.where(amax > 0, step, 1.0)
                out[i, :, a : a + GROUP] = torch.round(w / step) * step
        return out
    at = s["host_offsets"]
    y = torch.zeros((c["rows"], n), dtype=torch.float64, device=DEV)
    nibble = [0, 4, 1, 5, 2, 6, 3, 7]  # of weight j in its word
    for i in range(c["experts"]):
        if at[i] == at[i + 1]:
            continue
        words = s["data"][i].view(torch.int32).long()  # [tiles, blocks, 2 x 8 rows x 4 parts x 4 words]
        tiles, blocks, _ = words.shape
        q = torch.stack([(words >> (4 * j)) & 15 for j in nibble], -1).double() - 8.0
        q = q.view(tiles, blocks, 16, GROUP) * s["scales"][i].double()[..., None]
        w = q.transpose(1, 2).reshape(tiles * 16, blocks * GROUP)[:n, :k]
        y[at[i] : at[i + 1]] = s["x"][at[i] : at[i + 1]].double() @ w.t()
    return y
