"""8-bit blocks and the products on them, against 64-bit statements of the same operators.

Quantization is exact up to one defined rounding, so its bytes are compared for equality.  A product's terms (8-bit
values and powers of two) are exact in fp32, so a sum of K of them is off by at most K 2^-23 times the sum of their
magnitudes, for additions that round or truncate in any order, and the result is rounded once to its type.
"""
import numpy as np
import pytest

from gpu_helpers import require_gpu
from moe_oracle import (dequantize, doubles, half_ulp, quantize, quantize_blocks, quantize_columns, smallest,
                        unpack_scales)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import fp8  # noqa: E402

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def activations(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.exp(torch.randn(shape, generator=g) * 1.5 - 3.0) * torch.sign(torch.randn(shape, generator=g))
    x[torch.rand(shape, generator=g) < 0.005] = 0.0
    return x.to(dtype).cuda()


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def check_matrix(m, values, exponents, cols):
    """A Matrix's values, scales and padding against the statement's."""
    rows = values.shape[0]
    assert m.rows == rows and m.cols == cols
    got = m.values().float().cpu().numpy()
    assert np.array_equal(got.astype(np.float64), values, equal_nan=True)
    assert np.array_equal(np.signbit(got[values == 0]), np.signbit(values[values == 0]))
    blocks = m.data.shape[1] // 128
    scales = m.scales.cpu().numpy()
    assert np.array_equal(unpack_scales(scales, blocks), exponents)
    assert np.all(unpack_scales(scales, scales.shape[0] * 4)[:, blocks:] == 0)
    assert not m.data[:, cols:].any().item()


def test_scale_values():
    """Every scale byte, in words of which the last CTA has only a part: 2^(byte - 127), 255 a NaN."""
    for words in (1, 64, 257, 5000):
        data = (torch.arange(4 * words) % 256).to(torch.uint8).view(1, words, 4).cuda()
        m = fp8.Matrix(torch.zeros((words, 128), dtype=torch.uint8, device="cuda"), data, cols=100)
        got = doubles(m.scale_values())
        expect = np.exp2((np.arange(4 * words) % 256).reshape(1, words, 4) - 127.0)
        expect[expect == 2.0**128] = np.nan
        assert got.shape == expect.shape and np.array_equal(got, expect, equal_nan=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again = m.scale_values(stream=side)
        side.synchronize()
        assert np.array_equal(doubles(again), expect, equal_nan=True)
    with pytest.raises(TypeError):
        fp8.Matrix(torch.zeros((1, 128), dtype=torch.uint8), torch.zeros((1, 1, 4), dtype=torch.uint8), 3).scale_values()
    assert fp8.quantize(torch.zeros((0, 200), device="cuda")).scale_values().shape == (1, 0, 4)
    assert fp8.quantize(torch.zeros((0, 200), device="cuda")).values().shape == (0, 200)


SHAPES = [(1, 1), (1, 128), (2, 127), (5, 129), (33, 512), (64, 640), (7, 1000), (131, 2048), (3, 7168)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, fmt):
    wide = activations((rows, cols + (rows % 3) * 5), rows * 7 + cols, dtype)
    x = wide[:, :cols]
    check_matrix(fp8.quantize(x, fmt), *quantize(doubles(x), fmt), cols)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_every_bf16_pattern(fmt):
    """All 65,536 patterns, blocks of neighbours and of strangers: subnormals, the largest values, NaN, Inf, -0."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    for b in (bits, bits[torch.randperm(1 << 16, generator=torch.Generator().manual_seed(1))]):
        x = b.view(torch.bfloat16).view(64, 1024).cuda()
        check_matrix(fp8.quantize(x, fmt), *quantize(doubles(x), fmt), 1024)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_scale_boundaries(fmt):
    """Largest magnitudes on either side of MAX 2^s, ties between neighbouring 8-bit values, extreme exponents."""
    top = 448.0 if fmt == "e4m3" else 57344.0
    rows = []
    for s in (-140, -127, -126, -20, -1, 0, 1, 30, 100):
        for f in (1.0, np.nextafter(np.float32(1), np.float32(2)), np.nextafter(np.float32(1), np.float32(0))):
            a = np.float32(top * float(f) * 2.0 ** s) if s > -140 else np.float32(2.0 ** -149)
            r = np.linspace(-float(a), float(a), 128).astype(np.float32)
            r[:8] = a * np.array([1, 0.5, 17 / 448, 17.5 / 448, 18 / 448, 2.0 ** -16, 2.0 ** -17, 3 * 2.0 ** -18], np.float32)
            rows.append(r)
    x = torch.from_numpy(np.stack(rows)).cuda()
    check_matrix(fp8.quantize(x, fmt), *quantize(doubles(x), fmt), 128)


COLUMN_CASES = [((1, 0, 2) * 110, 20), ((5,), 3), ((128,), 128), ((0, 300, 0), 33), ((1, 127, 129, 256), 70), ((40,) * 9, 257), ((0, 0), 16)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,cols", COLUMN_CASES)
def test_quantize_columns(counts, cols, dtype, fmt):
    offsets = starts(counts)
    rows = int(offsets[-1])
    x = activations((rows, cols + 3), rows + cols, dtype)[:, :cols]
    m = fp8.quantize_columns(x, torch.from_numpy(offsets).cuda(), fmt)
    values, exponents, block_starts = quantize_columns(doubles(x), offsets, fmt)
    assert np.array_equal(m.offsets.cpu().numpy(), block_starts)
    check_matrix(m, values, exponents, values.shape[1])


def test_quantize_columns_leaves_rows_without_a_group():
    """Rows behind the last group are in no block, whatever they hold."""
    x = activations((500, 64), 1)
    x[300:] = float("nan")
    offsets = np.array([0, 130, 300], np.int32)
    m = fp8.quantize_columns(x, torch.from_numpy(offsets).cuda())
    v, s, b = quantize_columns(doubles(x)[:300], offsets, "e4m3")
    n = b[-1]
    assert np.array_equal(m.offsets.cpu().numpy(), b)
    assert np.array_equal(m.values().float().cpu().numpy()[:, :n * 128], v[:, :n * 128])
    assert np.array_equal(unpack_scales(m.scales.cpu().numpy(), n), s[:, :n])
    assert not m.data[:, n * 128:].any().item()


def test_quantize_columns_without_offsets():
    x = activations((300, 50), 2)
    m = fp8.quantize_columns(x)
    values, exponents, block_starts = quantize_columns(doubles(x), np.array([0, 300]), "e4m3")
    assert m.offsets.tolist() == block_starts.tolist()
    check_matrix(m, values, exponents, values.shape[1])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (3, 130, 257), (2, 128, 128), (1, 300, 64), (200, 700)])
def test_quantize_weight(shape, dtype, fmt):
    w = activations(shape, sum(shape), dtype)
    m, t = fp8.quantize_weight(w, fmt)
    assert m.data.dim() == w.dim() == t.data.dim()
    n, k = shape[-2:]
    for e in range(shape[0] if len(shape) == 3 else 1):
        we = doubles(w[e] if len(shape) == 3 else w)
        wide = np.zeros((-(-n // 128) * 128, -(-k // 128) * 128))
        wide[:n, :k] = we
        nb, kb = wide.shape[0] // 128, wide.shape[1] // 128
        blocks = wide.reshape(nb, 128, kb, 128).transpose(0, 2, 1, 3).reshape(nb, kb, 128 * 128)
        v, s = quantize_blocks(blocks, fmt)
        v = v.reshape(nb, kb, 128, 128).transpose(0, 2, 1, 3).reshape(wide.shape)[:n, :k]
        pick = (lambda a: a[e]) if len(shape) == 3 else (lambda a: a)
        check_matrix(fp8.Matrix(pick(m.data), pick(m.scales), k, fmt), v, np.repeat(s, 128, 0)[:n], k)
        check_matrix(fp8.Matrix(pick(t.data), pick(t.scales), n, fmt), v.T, np.repeat(s.T, 128, 0)[:k], n)
    alone, none = fp8.quantize_weight(w, fmt, transposed=False)
    assert none is None and torch.equal(alone.data, m.data) and torch.equal(alone.scales, m.scales)


def check_product(got, a, b, terms, dtype):
    """got against a @ b.T of doubles, with the sum of |terms| and `terms` additions."""
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    err = terms * 2.0 ** -23 * size
    bound = err + half_ulp(dtype) * (np.abs(want) + err) + smallest(dtype)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


# rows of each group, n, k: single rows, odd sizes, empty groups, tiles that end inside, many groups
PRODUCT_CASES = [((1,), 1, 1), ((1,), 128, 128), ((3,), 130, 257), ((0, 5, 0, 1), 64, 512), ((128, 256), 256, 384),
                 ((100, 0, 300, 17, 129), 200, 1000), ((1,) * 20, 136, 700), ((700, 3), 513, 896), ((9, 20), 384, 4100),
                 ((2, 0, 1), 129, 7168), ((33,) * 40, 260, 130)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,n,k", PRODUCT_CASES)
def test_matmul(counts, n, k, out_dtype):
    offsets = starts(counts)
    rows, e = int(offsets[-1]), len(counts)
    x = activations((rows, k), n + k)
    w = (torch.randn((e, n, k), generator=torch.Generator().manual_seed(k)) * 0.02).cuda()
    a, (b, _) = fp8.quantize(x), fp8.quantize_weight(w, transposed=False)
    got = fp8.matmul(a, b, torch.from_numpy(offsets).cuda(), out_dtype)
    assert got.dtype == out_dtype
    av, bv = dequantize(a), dequantize(b)
    for g in range(e):
        s = slice(offsets[g], offsets[g + 1])
        check_product(doubles(got[s]), av[s], bv[g], k, out_dtype)


@pytest.mark.parametrize("a_fmt,b_fmt", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("rows", [2, 70, 300])
def test_matmul_formats(a_fmt, b_fmt, rows):
    n, k = 140, 650
    a, b = fp8.quantize(activations((rows, k), 1), a_fmt), fp8.quantize(activations((n, k), 2), b_fmt)
    got = fp8.matmul(a, b, out_dtype=torch.float32)
    check_product(doubles(got), dequantize(a), dequantize(b), k, torch.float32)


def test_matmul_identity_places_every_value():
    """Powers of two that differ for every output: a wrong place, block or scale shows as a wrong value."""
    k = n = 512
    eye = torch.eye(k, device="cuda")
    a = fp8.quantize(eye * torch.exp2((torch.arange(k, device="cuda") % 23 - 11).float())[:, None])
    x = torch.exp2(((torch.arange(n, device="cuda")[:, None] * 7 + torch.arange(k, device="cuda") * 3) % 13).float())
    b = fp8.quantize(x)
    got = fp8.matmul(a, b, out_dtype=torch.float32)
    assert np.array_equal(doubles(got), dequantize(a) @ dequantize(b).T)


def test_matmul_many_row_tiles_and_wide_scales():
    """Scales far apart from block to block and row to row (2^-60 .. 2^60), more than one wave of tiles."""
    g = torch.Generator().manual_seed(3)
    rows, n, k = 5000, 1100, 640
    x = activations((rows, k), 4) * torch.exp2(torch.randint(-30, 30, (rows, k // 128), generator=g).float()).repeat_interleave(128, 1).cuda()
    w = activations((n, k), 5) * torch.exp2(torch.randint(-30, 30, (n, k // 128), generator=g).float()).repeat_interleave(128, 1).cuda()
    a, b = fp8.quantize(x), fp8.quantize(w)
    got = fp8.matmul(a, b, out_dtype=torch.float32)
    check_product(doubles(got), dequantize(a), dequantize(b), k, torch.float32)


@pytest.mark.parametrize("counts,n,k", [
    ((2048,), 2432, 300),             # 152 tiles of 128 x 256: one wave of single CTAs, two of pairs
    ((100,) * 38, 500, 260),          # 152 tiles of 128 x 128
    ((64,) * 3 + (0, 200), 2100, 520),  # groups above and below the average
    ((40,) * 3 + (0, 90), 300, 5000),   # blocks shared out, a group of two tiles, one of none
    ((3, 0, 1, 20), 257, 6000),         # the same with the smallest tiles
    ((1,) * 20, 130, 20000),            # parts of two tiles in one CTA
    ((1,) * 40, 500, 5000),             # 8 tiles more than SMs, shared out, and whole ones
    ((1,) * 30, 500, 5000),             # too many tiles to share out
    ((1,) * 300, 130, 140),           # more groups than CTAs
    ((256, 255, 257, 1, 511), 256, 128),  # tile ends on, before and after group ends, one block
    ((500,) * 6, 2050, 640),          # several bands of tiles, rows of out not whole 32-bit words apart
])
def test_matmul_cuts(counts, n, k):
    """Every way a product is cut into tiles, with groups that end inside them."""
    offsets = starts(counts)
    e = len(counts)
    x = activations((int(offsets[-1]), k), n)
    w = (torch.randn((e, n, k), generator=torch.Generator().manual_seed(n)) * 0.02).cuda()
    a, (b, _) = fp8.quantize(x), fp8.quantize_weight(w, transposed=False)
    got = doubles(fp8.matmul(a, b, torch.from_numpy(offsets).cuda(), torch.bfloat16))
    av, bv = dequantize(a), dequantize(b)
    for g in range(e):
        s = slice(offsets[g], offsets[g + 1])
        check_product(got[s], av[s], bv[g], k, torch.bfloat16)


def test_matmul_into_unaligned_rows():
    """Odd row widths: neighbouring rows of out start on and off word boundaries."""
    for n in (1, 31, 33, 127, 129, 255):
        a, b = fp8.quantize(activations((290, 200), n)), fp8.quantize(activations((n, 200), 1))
        check_product(doubles(fp8.matmul(a, b)), dequantize(a), dequantize(b), 200, torch.bfloat16)


def test_matmul_long_sums():
    """Many blocks in one sum, and many CTAs' parts in one tile."""
    for rows in (1, 40, 200):
        a, b = fp8.quantize(activations((rows, 40000), 1)), fp8.quantize(activations((70, 40000), 2))
        got = fp8.matmul(a, b, out_dtype=torch.float32)
        check_product(doubles(got), dequantize(a), dequantize(b), 40000, torch.float32)


@pytest.mark.parametrize("rows", [5, 300])
def test_matmul_extreme_scales(rows):
    """Scale bytes from 0 (2^-127) up, met by the other side's inverse so that the products are ordinary numbers."""
    g = torch.Generator().manual_seed(1)
    k, n = 640, 150
    e = torch.tensor([-127.0, -120.0, -60.0, 60.0, 110.0])
    x = torch.randint(-28, 29, (rows, k), generator=g) * torch.exp2(e + 4).repeat_interleave(128)
    w = torch.randint(-28, 29, (n, k), generator=g) * torch.exp2(-e - 10).repeat_interleave(128)
    x[:, ::128], w[:, ::128] = 28 * torch.exp2(e + 4), 28 * torch.exp2(-e - 10)  # (each block has its largest)
    a, b = fp8.quantize(x.cuda()), fp8.quantize(w.cuda())
    assert a.scales.min().item() == 0 and a.scales.max().item() == 127 + 110
    got = fp8.matmul(a, b, out_dtype=torch.float32)
    check_product(doubles(got), dequantize(a), dequantize(b), k, torch.float32)


def test_sizes_past_32_bit_offsets():
    """An output of more than 2^31 values, and 8-bit rows of more than 2^31 bytes."""
    rows, n = 50000, 45000
    a, b = fp8.quantize(activations((rows, 128), 1)), fp8.quantize(activations((n, 128), 2))
    got = fp8.matmul(a, b)
    assert got.numel() > 1 << 31
    av, bv = dequantize(a), dequantize(b)
    for r in (0, 1, rows // 2, rows - 1):
        check_product(doubles(got[r:r + 1]), av[r:r + 1], bv, 128, torch.bfloat16)
    del got
    x = torch.zeros((300001, 7168), dtype=torch.bfloat16, device="cuda")
    x[-1] = activations((7168,), 3, torch.bfloat16)
    q = fp8.quantize(x)
    last = fp8.quantize(x[-1:])
    assert q.data.numel() > 1 << 31 and torch.equal(q.data[-1], last.data[0])
    assert torch.equal(q.scales[:, -1], last.scales[:, 0]) and not q.data[:-1].any().item()
    c = fp8.quantize_columns(x)
    assert torch.equal(c.offsets, torch.tensor([0, -(-300001 // 128)], dtype=torch.int32, device="cuda"))
    got = c.values()[:, 300000].float() * torch.exp2(c.scales[300000 // 128 // 4, :, 300000 // 128 % 4].float() - 127)
    one = fp8.quantize_columns(x[-1:])
    assert torch.equal(got, one.values()[:, 0].float() * torch.exp2(one.scales[0, :, 0].float() - 127))


@pytest.mark.parametrize("rows", [3, 400])
def test_matmul_keeps_infinity_and_nan_in_their_rows(rows):
    x = activations((rows, 384), 6)
    x[1, 200] = float("nan")
    x[2, 300] = float("inf")
    w = activations((150, 384), 7).abs() + 0.01
    clean = x.clone()
    clean[1:3] = 0
    b = fp8.quantize(w)
    got, want = fp8.matmul(fp8.quantize(x, "e5m2"), b), fp8.matmul(fp8.quantize(clean, "e5m2"), b)
    assert got[1].isnan().all() and got[2].isinf().all()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert torch.equal(got[keep], want[keep])
    assert fp8.matmul(fp8.quantize(x), b)[1:3].isnan().all()  # e4m3 has no infinity: NaN


def test_matmul_rows_without_a_group_are_zero():
    a, b = fp8.quantize(activations((600, 256), 1)), fp8.quantize_weight(activations((2, 100, 256), 2))[0]
    a.data[300:] = 0x7F  # NaN: never read into a result
    offsets = torch.tensor([0, 77, 300], dtype=torch.int32, device="cuda")
    got = fp8.matmul(a, b, offsets)
    av, bv = dequantize(a), dequantize(b)
    check_product(doubles(got[:77]), av[:77], bv[0], 256, torch.bfloat16)
    check_product(doubles(got[77:300]), av[77:300], bv[1], 256, torch.bfloat16)
    assert not got[300:].float().abs().sum().item()


def test_matmul_no_rows():
    b = fp8.quantize(activations((64, 128), 2))
    a = fp8.quantize(torch.empty((0, 128), device="cuda"))
    assert fp8.matmul(a, b).shape == (0, 64)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,n,k", [((1,), 1, 1), ((128,), 128, 128), ((0, 300, 0), 33, 70), ((1, 127, 129, 512), 257, 130),
                                        ((40,) * 9, 64, 640), ((1500, 700), 300, 513), ((0, 0), 5, 9), ((6,) * 70, 130, 20)])
def test_weight_grad(counts, n, k, out_dtype):
    offsets = starts(counts)
    rows, e = int(offsets[-1]), len(counts)
    at = torch.from_numpy(offsets).cuda()
    dy, x = fp8.quantize_columns(activations((rows, n), 1), at, "e5m2"), fp8.quantize_columns(activations((rows, k), 2), at)
    got = fp8.weight_grad(dy, x, out_dtype)
    assert got.shape == (e, n, k) and got.dtype == out_dtype
    dv, xv, b = dequantize(dy), dequantize(x), dy.offsets.tolist()
    for g in range(e):
        s = slice(b[g] * 128, b[g + 1] * 128)
        check_product(doubles(got[g]), dv[:, s], xv[:, s], max(1, b[g + 1] - b[g]) * 128, out_dtype)


def test_backward_matches_differences():
    """The three products against differences of <matmul(x, w), g> along random directions.

    Values are whole numbers up to 7 (exact in e4m3 with the blocks' scales, sums exact in fp32), so the product is
    exactly bilinear and every difference equals the gradient's product with the direction."""
    g = torch.Generator().manual_seed(5)
    rows, n, k, e = 300, 140, 260, 3
    offsets = torch.tensor([0, 100, 110, 300], dtype=torch.int32, device="cuda")

    def whole(*shape, top=3):
        return torch.randint(-top, top + 1, shape, generator=g).float().cuda()

    x, w, gy = whole(rows, k), whole(e, n, k), whole(rows, n)
    dx_dir, dw_dir = whole(rows, k), whole(e, n, k)

    def loss(x_, w_):
        y = fp8.matmul(fp8.quantize(x_), fp8.quantize_weight(w_)[0], offsets, torch.float32)
        return float((doubles(y) * doubles(gy)).sum())

    _, w_t = fp8.quantize_weight(w)
    dx = fp8.matmul(fp8.quantize(gy), w_t, offsets, torch.float32)
    dw = fp8.weight_grad(fp8.quantize_columns(gy, offsets), fp8.quantize_columns(x, offsets), torch.float32)
    assert (loss(x + dx_dir, w) - loss(x - dx_dir, w)) / 2 == float((doubles(dx) * doubles(dx_dir)).sum())
    assert (loss(x, w + dw_dir) - loss(x, w - dw_dir)) / 2 == float((doubles(dw) * doubles(dw_dir)).sum())


def test_same_bits_every_time():
    offsets = torch.tensor([0, 5, 9, 40], dtype=torch.int32, device="cuda")
    a, (b, _) = fp8.quantize(activations((40, 4096), 1)), fp8.quantize_weight(activations((3, 300, 4096), 2))
    first = fp8.matmul(a, b, offsets)
    for _ in range(5):
        assert torch.equal(first, fp8.matmul(a, b, offsets))


def test_captured_in_a_graph():
    offsets = torch.tensor([0, 100, 333], dtype=torch.int32, device="cuda")
    x, (w, _) = activations((333, 300), 1), fp8.quantize_weight(activations((2, 200, 300), 2))

    def step():
        y = fp8.matmul(fp8.quantize(x), w, offsets)
        c = fp8.quantize_columns(x, offsets)
        return y, fp8.weight_grad(c, c)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    x.copy_(activations((333, 300), 9))
    offsets.copy_(torch.tensor([0, 3, 250]))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    del g


def test_on_another_stream():
    x, w = activations((200, 300), 1), fp8.quantize(activations((100, 300), 2))
    want = fp8.matmul(fp8.quantize(x), w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fp8.matmul(fp8.quantize(x, stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_group_starts_out_of_range_are_reported():
    """Starts that run past the rows or backwards: nothing outside the rows is read or written, and it is reported."""
    a, b = fp8.quantize(activations((200, 128), 1)), fp8.quantize_weight(activations((3, 64, 128), 2))[0]
    for bad in ([0, 100, 400, 500], [0, 150, 60, 200], [-50, 10, 20, 200]):
        at = torch.tensor(bad, dtype=torch.int32, device="cuda")
        fp8.matmul(a, b, at)
        assert zc.status(reset=True) == zc.ZC_ERR_CORRUPT, bad
        fp8.quantize_columns(activations((200, 64), 3), at)
        assert zc.status(reset=True) == zc.ZC_ERR_CORRUPT, bad


def test_refusals():
    x = activations((8, 256), 1)
    a, b = fp8.quantize(x), fp8.quantize(activations((4, 256), 2))
    at = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: fp8.quantize(x.cpu()), lambda: fp8.quantize(x.double()), lambda: fp8.matmul(a, b, at.long()),
                 lambda: fp8.matmul(a, b, out_dtype=torch.float16), lambda: fp8.quantize_columns(x, at.float()),
                 lambda: fp8.Matrix(a.data.view(torch.int8), a.scales, 256)):
        with pytest.raises(TypeError):
            call()
    two = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: fp8.quantize(x, "e3m4"), lambda: fp8.quantize(x[0]), lambda: fp8.quantize(x[:, :0]),
                 lambda: fp8.matmul(a, fp8.quantize(activations((4, 255), 2))), lambda: fp8.matmul(a, b, two),
                 lambda: fp8.Matrix(a.data, a.scales, 300), lambda: fp8.Matrix(a.data, a.scales[:, :4], 256),
                 lambda: fp8.Matrix(a.data[:, ::2], a.scales, 128), lambda: fp8.weight_grad(a, b),
                 lambda: fp8.quantize_weight(x[0]), lambda: fp8.matmul(a, b, at[:1])):
        with pytest.raises(ValueError):
            call()
