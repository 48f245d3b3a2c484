"""A mixture-of-experts layer whose exchanges are compressed, forward and backward, on one GPU.

A router chooses each token's experts and their weights (``moe.route``); tokens are sorted by expert into a send buffer
(``moe.dispatch``); the buffer crosses the all-to-all compressed, with the
transfer itself taken out (``binding.loopback`` compresses and decodes in one launch); the experts' two products run in
8-bit blocks (``fp8``); their outputs cross back the same way and are added with the router's weights (``moe.combine``).
The backward step sends the gradients through the same exchanges in the other direction, and the weights' gradients,
with that of the loss that keeps the experts evenly used (``moe.balance``), to the router's logits.

    python examples/expert_layer.py [--tokens 4096] [--hidden 2048] [--inner 1024] [--experts 16] [--k 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import fp8, moe  # noqa: E402


class ExpertLayer:
    """out[t] = sum over a token's experts of weight * relu(x[t] w1[e]^T) w2[e]^T."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor):
        """w1 [experts, inner, hidden] and w2 [experts, hidden, inner], bfloat16."""
        self.experts = w1.shape[0]
        self.w1, self.w1_t = fp8.quantize_weight(w1)
        self.w2, self.w2_t = fp8.quantize_weight(w2)
        self.exchanged, self.sent = 0, []  # bytes of rows exchanged, and the lengths of their streams

    def exchange(self, rows: torch.Tensor) -> torch.Tensor:
        """The rows as they arrive: compressed, sent, decompressed."""
        _, length, values = zc.loopback(rows)
        self.exchanged += rows.numel() * 2
        self.sent.append(length)
        return values.view(torch.bfloat16).view(rows.shape)

    def forward(self, x, experts_of, weights):
        rows, plan = moe.dispatch(x, experts_of, self.experts)
        rows = self.exchange(rows)
        h = torch.relu_(fp8.matmul(fp8.quantize(rows), self.w1, plan.offsets))
        y = self.exchange(fp8.matmul(fp8.quantize(h), self.w2, plan.offsets))
        self.saved = rows, h, y, plan, weights
        return moe.combine(y, weights, plan)

    def backward(self, d_out, out_dtype=torch.bfloat16):
        """(dx, d_weights, dw1, dw2) of the last forward; the weights' gradients in `out_dtype`."""
        rows, h, y, plan, weights = self.saved
        dy, d_weights = moe.combine_grad(d_out, y, weights, plan)
        dy = self.exchange(dy)
        dh = fp8.matmul(fp8.quantize(dy), self.w2_t, plan.offsets).mul_(h > 0)
        dw2 = fp8.weight_grad(fp8.quantize_columns(dy, plan.offsets), fp8.quantize_columns(h, plan.offsets), out_dtype)
        dw1 = fp8.weight_grad(fp8.quantize_columns(dh, plan.offsets), fp8.quantize_columns(rows, plan.offsets), out_dtype)
        d_rows = self.exchange(fp8.matmul(fp8.quantize(dh), self.w1_t, plan.offsets))
        return moe.dispatch_grad(d_rows, plan), d_weights, dw1, dw2

    def ratio(self) -> float:
        """Bytes of rows over bytes sent, of all exchanges so far."""
        return self.exchanged / max(1, sum(int(n.item()) for n in self.sent))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("k", 4)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    layer = ExpertLayer(normal(a.experts, a.inner, a.hidden, scale=a.hidden ** -0.5),
                        normal(a.experts, a.hidden, a.inner, scale=a.inner ** -0.5))
    x, d_out = normal(a.tokens, a.hidden), normal(a.tokens, a.hidden, scale=1e-3)
    logits = torch.randn((a.tokens, a.experts), generator=g, device="cuda")
    d_loss = torch.full((), 0.01, device="cuda")

    def step():
        weights, experts_of = moe.route(logits, a.k)
        balance = moe.balance(logits, experts_of)
        out = layer.forward(x, experts_of, weights)
        dx, d_weights, dw1, dw2 = layer.backward(d_out)
        return out, balance, dx, dw1, dw2, moe.route_grad(d_weights, logits, experts_of, balance=(d_loss, balance))

    balance = step()[1]
    layer.exchanged, layer.sent = 0, []
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    step()
    end.record()
    if (code := zc.status()) != zc.ZC_OK:
        raise zc.ZcError(code, "expert layer")
    flop = 3 * 2 * 2 * a.tokens * a.k * a.hidden * a.inner
    ms = begin.elapsed_time(end)
    print(f"forward and backward of {a.tokens} tokens x {a.k} of {a.experts} experts: {ms:.2f} ms, "
          f"{flop / ms / 1e9:.0f} TFLOP/s; rows exchanged compress {layer.ratio():.3f}x; balance loss {float(balance.loss):.3f}")


if __name__ == "__main__":
    main()
