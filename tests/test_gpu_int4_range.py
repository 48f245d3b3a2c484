"""Products on 4-bit weights with rows of very small values and large scales, and of very large ones and small scales: every
bit of x counts as long as the result is not itself near the end of fp32's range, nor a block's sum above 2^133.

A value of x is the sum of up to three parts of eight bits, each exact, so a single weight gives x times its value
exactly; sums are held to the bound of the products' other tests.
"""
import numpy as np
import pytest

import router_oracle as oracle
from gpu_helpers import require_gpu
from test_gpu_int4 import check_product, made

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import int4  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def small(rows, k, dtype, low, high, seed):
    """Values of random bits and of magnitudes from 2^low to 2^high, below the smallest normal number as well."""
    g = torch.Generator().manual_seed(seed)
    v = (1 + torch.rand((rows, k), generator=g, dtype=torch.float64)) * 2.0 ** torch.randint(low, high, (rows, k), generator=g).double()
    return (v * (torch.randint(0, 2, (rows, k), generator=g) * 2 - 1)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 6])
def test_every_bit_of_small_values_counts(rows, dtype):
    """Single weights of 2^100."""
    k = 256
    q = np.zeros((k, 2, 128), dtype=np.int64)
    q.reshape(k, k)[np.arange(k), np.arange(k)] = 1
    d, s = oracle.pack(q, np.full((k, 2), 2.0 ** 100))
    m = int4.Matrix(torch.from_numpy(d).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(), k, k)
    x = small(rows, k, dtype, -149 if dtype == torch.float32 else -133, -100, rows)
    x[0, 0], x[0, 1] = torch.finfo(dtype).smallest_normal / 2, -torch.finfo(dtype).smallest_normal
    x[1, 0] = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    got = int4.matmul(x.cuda(), m, None, torch.float32)
    assert torch.equal(got.cpu().double(), x.double() * 2.0 ** 100)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low,high", [(-126, -110), (-135, -126)])
def test_sums_of_small_values(low, high, dtype):
    m, values = made(0, 100, 700, 3)
    m = int4.Matrix(m.data, m.scales * 2.0 ** 110, 100, 700)
    check_product(small(5, 700, dtype, low, high, 4).cuda(), m, values * 2.0 ** 110, None, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("count", [4, 9, 18])
def test_sums_of_large_values(count, dtype):
    """Values next to 2^127 whose leading eight bits are a one and zeros, all bits behind them set, times 7: a block's sum, up
    to 126 times 2^127, is far above fp32's largest number until its scale is applied."""
    k = 256
    q = np.zeros((20, 2, 128), dtype=np.int64)
    q[:, :, 3:3 + 7 * count:7] = 7
    d, s = oracle.pack(q, np.full((20, 2), 2.0 ** -60))
    m = int4.Matrix(torch.from_numpy(d).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(), 20, k)
    x = torch.full((4, k), 2.0 ** 127 * (1 + 65535 / 2 ** 23), dtype=torch.float64).to(dtype).cuda()
    x[1], x[2, ::2], x[3] = -x[1], -x[2, ::2], x[3] / 2
    check_product(x, m, oracle.weight_values(q, np.full((20, 2), 2.0 ** -60), k)[None], None, torch.float32)
