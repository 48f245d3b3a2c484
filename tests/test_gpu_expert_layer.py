"""The expert layer of examples/: sorted, compressed, multiplied in 8-bit blocks, brought back, and its gradients.

The inputs are small whole numbers and halves that every rounding on the way keeps (8-bit values with power-of-two
scales, bfloat16, sums in fp32), so the layer must equal the dense layer in 64 bits exactly, dropped slots included.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import expert_layer  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def sparse(rng, experts, n, k, per_row):
    """[experts, n, k] of -1, 0, 1 with per_row nonzeros a row, at most about as many a column."""
    w = np.zeros((experts, n, k))
    for e in range(experts):
        for j in range(per_row):
            cols = np.concatenate([rng.permutation(k) for _ in range(-(-n // k))])[:n]
            w[e, np.arange(n), cols] = rng.choice([-1.0, 1.0], n)
    return w


@pytest.mark.parametrize("tokens,k,experts,hidden,inner", [(1, 2, 4, 128, 64), (60, 3, 5, 200, 136), (300, 2, 3, 136, 264)])
def test_layer_equals_the_dense_layer(tokens, k, experts, hidden, inner):
    rng = np.random.default_rng(tokens)
    w1, w2 = sparse(rng, experts, inner, hidden, 2), sparse(rng, experts, hidden, inner, 2)
    x = rng.integers(-2, 3, (tokens, hidden)).astype(np.float64)
    d_out = rng.integers(-1, 2, (tokens, hidden)).astype(np.float64)
    ids = np.stack([rng.permutation(experts)[:k] for _ in range(tokens)])
    ids[rng.random(ids.shape) < 0.2] = -1
    weights = rng.choice([0.5, 1.0], ids.shape)

    def gpu(a, dtype=torch.bfloat16):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()

    zc.status(reset=True)
    layer = expert_layer.ExpertLayer(gpu(w1), gpu(w2))
    out = layer.forward(gpu(x), gpu(ids, torch.int64), gpu(weights, torch.float32))
    dx, d_weights, dw1, dw2 = layer.backward(gpu(d_out), torch.float32)
    assert zc.status(reset=True) == zc.ZC_OK and layer.ratio() > 0

    want = {"out": np.zeros_like(x), "dx": np.zeros_like(x), "d_weights": np.zeros_like(weights),
            "dw1": np.zeros_like(w1), "dw2": np.zeros_like(w2)}
    for t in range(tokens):
        for j in range(k):
            e, c = ids[t, j], weights[t, j]
            if e < 0:
                continue
            h = np.maximum(w1[e] @ x[t], 0)
            y = w2[e] @ h
            want["out"][t] += c * y
            want["d_weights"][t, j] = d_out[t] @ y
            dh = (w2[e].T @ (c * d_out[t])) * (h > 0)
            want["dw2"][e] += np.outer(c * d_out[t], h)
            want["dw1"][e] += np.outer(dh, x[t])
            want["dx"][t] += w1[e].T @ dh
    for name, got in (("out", out), ("dx", dx), ("d_weights", d_weights), ("dw1", dw1), ("dw2", dw2)):
        assert np.array_equal(got.double().cpu().numpy(), want[name]), name


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer.py"), "--tokens", "512", "--hidden",
                        "512", "--inner", "256"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "rows exchanged compress" in r.stdout
