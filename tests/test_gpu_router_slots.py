"""Slots whose expert the token may not use (a logit of -infinity): they take no part in a gradient, whatever stands in
their place."""
import numpy as np
import pytest

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import moe  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("tokens,experts,k", [(9, 20, 3), (7, 50, 5), (5, 120, 40), (6, 200, 8), (4, 300, 8), (3100, 200, 8)])
def test_slots_that_may_not_be_used(tokens, experts, k, score, normalize, dtype):
    g = torch.Generator().manual_seed(tokens + k)
    x = torch.randn((tokens, experts), generator=g).to(dtype)
    ids = torch.rand((tokens, experts), generator=g).argsort(1)[:, :k].int()  # k of them, each once
    dw = torch.randn((tokens, k), generator=g)
    for j, v in ((0, np.nan), (1, np.inf), (2, -np.inf)):
        x.scatter_(1, ids[:, j:j + 1].long(), -np.inf)
        dw[:, j] = v
    x[3] = -np.inf  # padding
    without = torch.where(torch.arange(k) < 3, -1, ids).int()
    x, dw, ids, without = x.cuda(), dw.cuda(), ids.cuda(), without.cuda()
    b = moe.balance(x, without, score)
    for balance in (None, (torch.ones((), device="cuda"), b)):
        got = moe.route_grad(dw, x, ids, score, normalize, balance=balance)
        assert torch.isfinite(got).all() and (got[x == -np.inf] == 0).all()
        assert torch.equal(got, moe.route_grad(dw, x, without, score, normalize, balance=balance))
