"""Gradients of a router whose warps have several tokens one after the other, in every form of the kernels: what is
asked for a token ahead has to be that token's.

Compared with the formulas in 64 bits on all rows, to the bounds of the router's other tests: w (|g| + sum |g| w)
(2 D + 180) 2^-24 at every expert, D the row's spread of logits.
"""
import pytest

from gpu_helpers import require_gpu
from moe_oracle import half_ulp, smallest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import moe  # noqa: E402

E = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def shares(x, score):
    """Softmax of rows, or their sigmoids over their sum; zeros for rows of nothing but -infinity."""
    dead = (x == -INF).all(1, keepdim=True)
    x = torch.where(dead, 0.0, x if score == "softmax" else torch.nn.functional.logsigmoid(x))
    return torch.where(dead, 0.0, torch.softmax(x, 1))


def spread(x):
    finite = torch.isfinite(x)
    d = torch.where(finite, x, -INF).amax(1, keepdim=True) - torch.where(finite, x, INF).amin(1, keepdim=True)
    return torch.where(torch.isfinite(d), d, 0.0)


def weights_grad(dw, x, ids, score, normalize):
    """(gradient, its bound)."""
    kept = ids >= 0
    at = ids.long().clamp(min=0)
    g = torch.where(kept, dw.double(), 0.0)
    unit = (2 * spread(x) + 180) * E
    if (score, normalize) == ("softmax", False):
        p = shares(x, score)
        w = torch.where(kept, p.gather(1, at), 0.0)
        total = (g * w).sum(1, keepdim=True)
        bound = p * (g.abs() * w).sum(1, keepdim=True)
        want = -p * total
    else:
        top = torch.where(kept, x.gather(1, at), -INF)
        w = shares(top, score) if normalize else torch.sigmoid(top)
        total = (g * w).sum(1, keepdim=True) if normalize else torch.zeros_like(g[:, :1])
        want, bound = torch.zeros_like(x), torch.zeros_like(x)
    rest = torch.where(kept, 1 - torch.sigmoid(x.gather(1, at)), 0.0) if score == "sigmoid" else 1.0
    if (score, normalize) == ("softmax", False):
        total = torch.zeros_like(total)  # (taken off every expert above)
    want.scatter_add_(1, at, torch.where(kept, w * (g - total) * rest, 0.0))
    bound.scatter_add_(1, at, torch.where(kept, w * (g.abs() + (g.abs() * w).sum(1, keepdim=True)), 0.0))
    return want, bound * unit


def balance_grad(x, slope, score):
    p, slope = shares(x, score), slope.double()
    mean = (p * slope).sum(1, keepdim=True)
    want = p * (slope - mean)
    if score == "sigmoid":
        want = want * (1 - torch.sigmoid(x))
    return want, p * (slope + mean) * (2 * spread(x) + 180) * E


# Tokens side by side in a warp (64 and 128 experts), a row of 256 and one of 300 experts to a warp; a warp's slots of several
# tokens at once (256 and 300 experts, all scores but a softmax of the row).  On 152 SMs every warp has two at least.
CASES = [(40000, 64, 8), (20000, 128, 5), (10000, 256, 40), (80000, 256, 8), (40000, 300, 8), (3000, 300, 40)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("tokens,experts,k", CASES)
def test_a_warp_s_next_token(tokens, experts, k, score, normalize, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens + k)
    x = torch.randn((tokens, experts), generator=g, device="cuda") * 2
    x[torch.rand((tokens, experts), generator=g, device="cuda") < 0.1] = -INF
    x[torch.rand(tokens, generator=g, device="cuda") < 0.05] = -INF
    x = x.to(dtype)
    _, ids = moe.route(x, k, score, normalize)
    b = moe.balance(x, ids, score)
    dw = torch.randn((tokens, k), generator=g, device="cuda")
    d_loss = torch.full((), 3.0 * tokens, device="cuda")  # (as large a part as the weights')
    v = x.double()
    want, bound = weights_grad(dw, v, ids, score, normalize)
    want_loss, bound_loss = (t * 3.0 * tokens for t in balance_grad(v, b.slope, score))

    def held(got, want, bound):
        assert ((got.double() - want).abs() <= bound + half_ulp(dtype) * (want.abs() + bound) + smallest(dtype)).all()

    held(moe.route_grad(dw, x, ids, score, normalize), want, bound)
    held(moe.balance_grad(d_loss, x, b, score), want_loss, bound_loss)
    if (score, normalize) == ("softmax", False):  # one sum of both over the row, taken off every expert
        p = shares(v, score)
        bound = bound + p * 3.0 * tokens * (p * b.slope.double()).sum(1, keepdim=True) * (2 * spread(v) + 180) * E
    both, bound = want + want_loss, bound + bound_loss
    got = moe.route_grad(dw, x, ids, score, normalize, balance=(d_loss, b))
    held(got, both, bound + 2 * E * (both.abs() + bound))
    assert torch.equal(got, moe.route_grad(dw, x, ids, score, normalize, balance=(d_loss, b)))
