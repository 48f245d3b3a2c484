"""The experts' calls in the circumstances of a program: inputs written by the kernel just before, every number of
experts, rows and sizes at which a call takes another kernel.  What is only moved is compared bit for bit, what is
rounded to 8 bits as well; tolerances of sums as in test_gpu_moe.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import fp8, moe  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def routing(tokens, k, experts, seed, dropped=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
    return torch.where(torch.rand((tokens, k), generator=g, device="cuda") < dropped, -1, ids)


def values(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(
        a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ inputs written just before


@pytest.mark.parametrize("tokens,k,hidden", [(3000, 4, 1024), (3000, 4, 1021), (100, 4, 1024), (1, 8, 7168)])
def test_inputs_written_by_the_kernel_before(tokens, k, hidden):
    """Every call starts early; its inputs change with every round, written by the kernel before it, into the same
    buffers.  Nothing of an earlier round may show."""
    experts, rounds = 7, 12
    xs = [values((tokens, hidden), torch.bfloat16, i) for i in range(rounds)]
    routes = [routing(tokens, k, experts, i) for i in range(rounds)]
    ws = [values((tokens, k), torch.float32, 100 + i) for i in range(rounds)]
    b = fp8.quantize(values((96, hidden), torch.bfloat16, 50))
    x, ids, w = torch.empty_like(xs[0]), torch.empty_like(routes[0]), torch.empty_like(ws[0])
    rows = torch.empty((tokens * k, hidden), dtype=torch.bfloat16, device="cuda")

    def step(i, between):
        x.copy_(xs[i])
        ids.copy_(routes[i])
        between()
        r, plan = moe.dispatch(x, ids, experts)
        rows.copy_(r)
        w.copy_(ws[i])
        between()
        back = moe.combine(rows, w, plan)
        between()
        d_rows, d_w = moe.combine_grad(back, rows, w, plan)
        between()
        dx = moe.dispatch_grad(d_rows, plan)
        between()
        q = fp8.quantize(dx)
        between()
        y = fp8.matmul(q, b)
        between()
        c = fp8.quantize_columns(y)
        return [r, *plan, back, d_rows, d_w, dx, q.data, q.scales, y, c.data, c.scales, c.offsets]

    apart = [step(i, torch.cuda.synchronize) for i in range(rounds)]
    torch.cuda.synchronize()
    together = [step(i, lambda: None) for i in range(rounds)]
    for one, other in zip(apart, together):
        assert all(same_bits(a, b) for a, b in zip(one, other))
