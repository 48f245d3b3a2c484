"""Products on 4-bit weights of so many rows that offsets into x and into the results pass 32 bits, and the loss of a
router's batch, in graphs.

A product's rows are compared with those of a few rows alone, which are compared with 64 bits elsewhere: a block's sum of
whole numbers below 2^24 is exact, and with one block and scales of powers of two so is all that follows, up to the
one rounding, so that they have to be equal however the work is cut."""
import pytest

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import int4, moe  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def whole_numbers(groups, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    low, high = (torch.randint(1, 16, (groups, -(-n // 16), 1, 1024), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    scales = 2.0 ** torch.randint(-3, 1, (groups, -(-n // 16), 1, 16), generator=g, device="cuda").float()
    return int4.Matrix(low | high << 4, scales.bfloat16(), n, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_past_32_bit_offsets(dtype):
    """A million rows times matrices of 2100: 2.2 billion results, the last rows of no group."""
    rows, n = (1 << 20) + 5, 2100
    m = whole_numbers(3, n, 1)
    x = torch.randint(-8, 9, (rows, 128), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dtype)
    offsets = torch.tensor([0, 700001, 700001, rows - 3], dtype=torch.int32, device="cuda")
    y = int4.matmul(x, m, offsets, torch.bfloat16)
    assert (y[rows - 3:] == 0).all()
    for at, group in ((0, 0), (123457, 0), (700000 - 6, 0), (700001, 2), (1 << 20, 2), (rows - 10, 2)):
        one = int4.Matrix(m.data[group], m.scales[group], n, 128)
        assert torch.equal(y[at:at + 7][:min(7, rows - 3 - at)], int4.matmul(x[at:at + 7], one, None, torch.bfloat16)[:min(7, rows - 3 - at)])
    w = m.values()
    for at, c, group in ((0, 700001, 0), (700001, rows - 3 - 700001, 2)):  # exact in fp32, and rounded once
        for first in range(at, at + c, 100000):
            part = slice(first, min(at + c, first + 100000))
            want = x[part].float() @ w[group].t()  # (products and sums of whole numbers, exact in any order and in tf32)
            assert torch.equal(y[part], want.bfloat16())


def test_rows_past_32_bit_offsets():
    """Rows of x 600 million values apart."""
    m = whole_numbers(1, 70, 3)
    m = int4.Matrix(m.data[0], m.scales[0], 70, 128)
    buffer = torch.empty((9, 600_000_008), dtype=torch.bfloat16, device="cuda")
    x = buffer[:, 600_000_000 - 128:600_000_000]
    x.copy_(torch.randint(-8, 9, (9, 128), device="cuda"))
    assert torch.equal(int4.matmul(x, m), int4.matmul(x.contiguous(), m))


@pytest.mark.parametrize("tokens,experts", [(5000, 64), (3000, 300)])
def test_loss_of_two_kernels_in_graphs(tokens, experts):
    """Two graphs with workspaces from one pool and calls outside of them, on new contents."""
    def fill(x, seed):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))

    xs = [torch.zeros((tokens, experts), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kept, graphs = [], []

    def step(x):
        weights, ids = moe.route(x, 6, "sigmoid")
        return (weights, ids, *moe.balance(x, ids, "sigmoid"))

    step(xs[0])
    torch.cuda.synchronize()
    pool = torch.cuda.graph_pool_handle()
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            kept.append(step(x))
    for seed in range(3):
        for i, x in enumerate(xs):
            fill(x, 10 * seed + i)
        want = [step(x) for x in xs]
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(kept, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
