"""A router and its experts together, as they are used: logits, choice, balance loss, dispatch, products on 4-bit weights,
combine; and back to the logits.

Rows, weights and scales are whole numbers and powers of two, so that the experts' products are exact and only the router's
scores are rounded: what follows them is compared with 64 bits from the scores that the router gave.  combine's sum of k
products is off by k 2^-24 of their magnitudes and one rounding; a weight's gradient, a dot product over `hidden`, by
hidden 2^-24; the logits' gradient as in the router's own tests: w (|g| + sum |g| w) (2 D + 180) 2^-24.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import router_oracle as oracle
from gpu_helpers import require_gpu
from moe_oracle import doubles, half_ulp, smallest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import int4, moe  # noqa: E402

E = 2.0 ** -24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("tokens,experts,k,hidden,out", [(1, 8, 2, 256, 48), (5, 16, 4, 200, 130), (90, 12, 3, 384, 64), (400, 40, 6, 128, 33)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_and_experts(tokens, experts, k, hidden, out, score):
    rng = np.random.default_rng(tokens)
    x = rng.integers(-3, 4, (tokens, hidden)).astype(np.float64)
    # weights of which each group's largest is 7 times a power of two: kept exactly
    w = rng.integers(-7, 8, (experts, out, hidden)).astype(np.float64)
    w[:, :, ::128] = 7
    w *= 2.0 ** rng.integers(-3, 1, (experts, out, 1))
    logits = torch.randn((tokens, experts), generator=torch.Generator().manual_seed(tokens)).cuda() * 2
    logits[::7, 1:] = -np.inf  # some tokens with one expert only
    d_out = torch.from_numpy(rng.integers(-2, 3, (tokens, out)).astype(np.float32)).cuda()
    zc.status(reset=True)
    m = int4.quantize_weight(torch.from_numpy(w).float().cuda())
    assert np.array_equal(doubles(m.values()), w)

    weights, ids = moe.route(logits, k, score)
    b = moe.balance(logits, ids, score)
    rows, plan = moe.dispatch(torch.from_numpy(x).float().cuda(), ids, experts)
    y = int4.matmul(rows, m, plan.offsets)
    got = moe.combine(y, weights, plan)
    dy, dw = moe.combine_grad(d_out, y, weights, plan)
    d_loss = torch.full((), 0.5, device="cuda")
    d_logits = moe.route_grad(dw, logits, ids, score, balance=(d_loss, b))
    assert zc.status(reset=True) == zc.ZC_OK

    i, v, s = ids.cpu().numpy(), doubles(logits), doubles(weights)
    assert np.array_equal(i, oracle.choose(v, k))
    assert torch.equal(b.counts, plan.offsets[1:] - plan.offsets[:-1])
    products = np.einsum("eoh,th->teo", w, x)
    chosen = np.where((i >= 0)[..., None], products[np.arange(tokens)[:, None], np.maximum(i, 0)], 0.0)  # [tokens, k, out]
    want, size = (s[..., None] * chosen).sum(1), np.abs(s[..., None] * chosen).sum(1)
    assert (np.abs(doubles(got) - want) <= (k + 1) * E * size + smallest(torch.float32)).all()
    d = doubles(d_out)
    want_dw = (chosen * d[:, None, :]).sum(2)
    assert (np.abs(doubles(dw) - want_dw) <= (out + 1) * E * np.abs(chosen * d[:, None, :]).sum(2)).all()

    g = doubles(dw)
    want = oracle.route_grad(g, v, i, score, True) + oracle.balance_grad(0.5, v, doubles(b.slope), score)
    finite = np.where(np.isfinite(v), v, 0.0)
    spread = (finite.max(1) - finite.min(1))[:, None]
    ww, total = oracle.weights(v, i, score, True), np.zeros(v.shape)
    bound = np.where(i >= 0, ww * (np.abs(g) + (np.abs(g) * ww).sum(1, keepdims=True)), 0)
    for t in range(tokens):
        kept = i[t] >= 0
        np.add.at(total[t], i[t][kept], bound[t][kept])
    p, slope = oracle.probabilities(v, score), doubles(b.slope)
    total += 0.5 * p * (slope + (p * slope).sum(1, keepdims=True))
    assert (np.abs(doubles(d_logits) - want) <= total * (2 * spread + 182) * E + 2.0 ** -140).all()


def test_the_layer_captured_and_replayed():
    """The serving step of a batch in one graph, on new tokens and new routings."""
    tokens, experts, k, hidden = 16, 8, 2, 512
    m = int4.quantize_weight(torch.randn((experts, hidden, hidden), generator=torch.Generator().manual_seed(1)).bfloat16().cuda())
    x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    gate = torch.randn((hidden, experts), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()

    def step():
        weights, ids = moe.route(x @ gate, k)
        rows, plan = moe.dispatch(x, ids, experts)
        return moe.combine(int4.matmul(rows, m, plan.offsets), weights, plan), ids

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, ids = step()
    for seed in range(3):
        x.copy_(torch.randn((tokens, hidden), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        kept, chosen = out.clone(), ids.clone()
        want, again = step()
        assert torch.equal(chosen, again) and torch.equal(kept, want)


def test_example_routes_its_tokens():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer.py"), "--tokens", "300", "--hidden",
                        "512", "--inner", "256", "--experts", "8", "--k", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "balance loss" in r.stdout
