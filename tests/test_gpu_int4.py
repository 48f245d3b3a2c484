"""Weights in 4 bits and the products on them, against 64-bit statements of the same operators.

Rounding to 4 bits is decided exactly, so scales, records and values have to be equal.  A product's sum: a group's 128
products are exact (of up to three parts of x), and added in fp32 in an order and with a rounding that the matrix
instructions choose: below 2^-23 of the sum of magnitudes for each of at most 3 x 128 additions.  A group's sum is then
scaled and added, 2^-24 twice for each group and each slice of them (at most 8), and the parts are added at the end.  The
result is rounded once.  Whole numbers of small size are exact all the way and have to be equal.
"""
import numpy as np
import pytest

import router_oracle as oracle
from gpu_helpers import require_gpu
from moe_oracle import doubles, half_ulp, smallest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import int4  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def check_quantized(w, m):
    """w: the weights as doubles [experts, n, k] or [n, k]."""
    n, k = w.shape[-2:]
    data, scales = m.data.cpu().numpy(), doubles(m.scales)
    if w.ndim == 2:
        w, data, scales = w[None], data[None], scales[None]
    for e in range(len(w)):
        q, s = oracle.quantize(w[e])
        got_q, got_s, rest_q, rest_s = oracle.unpack(data[e], scales[e], n, k)
        assert np.array_equal(got_s, s, equal_nan=True)
        assert np.array_equal(got_q, q)
        assert (rest_q == 0).all() and (rest_s == 1).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (16, 128), (17, 129), (5, 1000), (100, 257), (3, 33, 384), (2, 16, 7), (4, 64, 136)])
def test_quantize_weight(shape, dtype):
    g = torch.Generator().manual_seed(sum(shape))
    w = (torch.randn(shape, generator=g) * 0.02).to(dtype)
    m = int4.quantize_weight(w.cuda())
    assert m.rows == shape[-2] and m.cols == shape[-1]
    check_quantized(doubles(w), m)
    for out in TYPES:
        v = m.values(out)
        assert v.shape == w.shape and v.dtype == out
        flat, many = doubles(w).reshape(-1, *shape[-2:]), v.cpu().reshape(-1, *shape[-2:])
        for e in range(len(flat)):
            q, s = oracle.quantize(flat[e])
            # q s has at most 11 significant bits, so it is exact in fp32 (fp16 underflows below its range)
            want = torch.from_numpy(oracle.weight_values(q, s, shape[-1])).float().to(out)
            assert torch.equal(many[e], want)


@pytest.mark.parametrize("dtype", TYPES)
def test_quotients_next_to_a_half(dtype):
    """Groups whose largest magnitude sets the scale, and values at, just below and just above every half step."""
    rows = []
    for amax in (7.0, 7.03125, 5.0, 1.75, 3.4375):
        s = oracle.bf16_at_least(amax / 7)
        v = [amax]
        for h in np.arange(0.5, 7.0, 1.0):
            t = torch.tensor(h * s, dtype=torch.float64).to(dtype)
            for step in (0, 1, -1):
                bits = t.view(torch.int16 if dtype != torch.float32 else torch.int32) + step
                v += [float(bits.view(dtype)), -float(bits.view(dtype))]
        rows.append((v + [0.0] * 128)[:128])
    w = torch.tensor(rows, dtype=torch.float64).to(dtype)
    check_quantized(doubles(w), int4.quantize_weight(w.cuda()))


def test_every_bfloat16_magnitude_as_the_largest():
    bits = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16)
    amax = bits.view(torch.bfloat16)
    w = torch.zeros((amax.numel(), 128), dtype=torch.bfloat16)
    w[:, 17] = -amax
    w[:, 100] = (amax.double() * 0.36).to(torch.bfloat16)
    m = int4.quantize_weight(w.cuda())
    s = doubles(m.scales).transpose(0, 2, 1).reshape(-1)[: amax.numel()]
    a = doubles(amax)
    unit = 2.0 ** np.maximum(np.frexp(s)[1] - 8, -133)
    assert (7 * s >= a).all()
    below = s - np.where(np.frexp(s)[0] == 0.5, np.maximum(unit / 2, 2.0 ** -133), unit)  # the next smaller value
    assert (7 * below < a).all()
    v = doubles(m.values())
    assert np.array_equal(v, np.rint(doubles(w) / s[:, None]) * s[:, None])


@pytest.mark.parametrize("dtype", TYPES)
def test_groups_of_zeros_and_of_what_is_not_finite(dtype):
    w = torch.zeros((20, 300), dtype=dtype)
    w[1, 130], w[2, 5], w[3, 299], w[4] = np.nan, np.inf, -np.inf, 1.0
    w[4, 0] = -0.0
    w[5, 0] = torch.finfo(dtype).max
    w[6, 0] = torch.finfo(dtype).smallest_normal / 4
    m = int4.quantize_weight(w.cuda())
    check_quantized(doubles(w), m)
    v = m.values()
    assert torch.isnan(v[1, 128:256]).all() and (v[1, :128] == 0).all() and torch.isnan(v[2, :128]).all()
    assert torch.isnan(v[3, 256:]).all() and (v[4, 1:] == 7 * 147 / 1024).all()  # 1 / 7 lies between 146 and 147 / 1024
    assert (v[0] == 0).all()


def made(groups, n, k, seed, whole=False):
    """Random 4-bit weights: (Matrix, values as doubles [groups, n, k]).  whole: scales of powers of two."""
    rng = np.random.default_rng(seed)
    data, scales, values = [], [], []
    for _ in range(max(1, groups)):
        q = rng.integers(-7, 8, (n, -(-k // 128), 128))
        q.reshape(n, -1)[:, k:] = 0
        s = 2.0 ** rng.integers(-2, 3, q.shape[:2]) if whole else rng.integers(128, 256, q.shape[:2]) * 2.0 ** rng.integers(-14, -10, q.shape[:2])
        d, sc = oracle.pack(q, s)
        data.append(d)
        scales.append(sc)
        values.append(oracle.weight_values(q, s, k))
    data, scales = np.stack(data), np.stack(scales)
    if not groups:
        data, scales = data[0], scales[0]
    m = int4.Matrix(torch.from_numpy(data).cuda(), torch.from_numpy(scales).to(torch.bfloat16).cuda(), n, k)
    return m, np.stack(values)


def expected(x, values, offsets):
    """(products, sums of magnitudes) in 64 bits."""
    y, a = np.zeros((len(x), values.shape[1])), np.zeros((len(x), values.shape[1]))
    for g in range(len(values)):
        rows = slice(offsets[g], offsets[g + 1])
        y[rows] = x[rows] @ values[g].T
        a[rows] = np.abs(x[rows]) @ np.abs(values[g]).T
    return y, a


def check_product(x, m, values, offsets, out_dtype=None):
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = int4.matmul(x, m, o, out_dtype)
    dtype = out_dtype or x.dtype
    assert y.dtype == dtype and y.shape == (x.shape[0], m.rows)
    want, size = expected(doubles(x), values, offsets or [0, x.shape[0]])
    bound = size * (3 * 128 * 2.0 ** -23 + (2 * -(-m.cols // 128) + 40) * 2.0 ** -24)
    assert (np.abs(doubles(y) - want) <= bound + half_ulp(dtype) * (np.abs(want) + bound) + smallest(dtype)).all()
    return y


# (rows, n, k): one of all, odd sizes, several blocks, slices and passes
SIZES = [(1, 1, 1), (1, 16, 128), (2, 130, 40), (1, 200, 1100), (7, 129, 2300), (8, 16, 1000), (9, 33, 257), (17, 48, 520), (33, 100, 300),
         (70, 40, 136), (5, 260, 9000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_one_matrix(rows, n, k, dtype):
    m, values = made(0, n, k, rows + n + k)
    x = torch.randn((rows, k), generator=torch.Generator().manual_seed(k)).to(dtype).cuda()
    for out in (None, torch.float32, torch.bfloat16, torch.float16):
        check_product(x, m, values, None, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts", [[3, 0, 1, 8], [0, 0, 5], [1] * 40, [20, 1, 0, 3, 9], [0, 0], [50, 2]])
@pytest.mark.parametrize("behind", [0, 3])
def test_groups(counts, behind, dtype):
    n, k = 70, 640
    m, values = made(len(counts), n, k, sum(counts) + len(counts))
    offsets = [0] + [int(v) for v in np.cumsum(counts)]
    rows = offsets[-1] + behind
    x = torch.randn((rows, k), generator=torch.Generator().manual_seed(rows)).to(dtype).cuda()
    if behind:
        x[-1] = np.nan  # a row of no group is not looked at
    y = check_product(torch.where(torch.isnan(x), 0, x), m, values, offsets)
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    z = int4.matmul(x, m, o)
    assert torch.equal(z, y) and (z[offsets[-1]:] == 0).all()


@pytest.mark.parametrize("groups", [1, 255, 256, 257, 1024])
def test_many_groups(groups):
    n, k = 16, 128
    few, values = made(min(groups, 37), n, k, groups)
    at = torch.arange(groups, device="cuda") % 37
    m, values = int4.Matrix(few.data[at], few.scales[at], n, k), values[at.cpu().numpy()]
    counts = np.random.default_rng(groups).integers(0, 3, groups)
    offsets = [0] + [int(v) for v in np.cumsum(counts)]
    x = torch.randn((offsets[-1], k), generator=torch.Generator().manual_seed(groups)).bfloat16().cuda()
    check_product(x, m, values, offsets)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,k", [(1, 300, 1024), (8, 17, 700), (13, 129, 2000), (40, 20, 5000)])
def test_whole_numbers_are_exact(rows, n, k, dtype):
    m, values = made(0, n, k, 3, whole=True)
    rng = np.random.default_rng(rows)
    x = rng.integers(-8, 9, (rows, k)).astype(np.float64)
    y = int4.matmul(torch.from_numpy(x).to(dtype).cuda(), m, None, torch.float32)
    assert np.array_equal(doubles(y), expected(x, values, [0, rows])[0])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_every_bit_of_x_counts(dtype):
    """x against single weights of 1: what bfloat16 does not hold comes back whole."""
    k = 256
    q = np.zeros((k, 2, 128), dtype=np.int64)
    q.reshape(k, k)[np.arange(k), np.arange(k)] = 1
    d, s = oracle.pack(q, np.ones((k, 2)))
    m = int4.Matrix(torch.from_numpy(d).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(), k, k)
    g = torch.Generator().manual_seed(5)
    x = (torch.randn((6, k), generator=g) * 2.0 ** torch.randint(-10, 10, (6, k), generator=g)).to(dtype).cuda()
    x[0, 0], x[0, 1], x[1, 5] = torch.finfo(dtype).max, -torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    if dtype == torch.float16:  # numbers too small to be normal, the smallest among them
        x[2] = torch.randint(-1023, 1024, (k,), generator=g).double().mul(2.0 ** -24).half()
    assert torch.equal(int4.matmul(x, m), x)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan_show_in_their_row_only(dtype):
    m, values = made(0, 40, 300, 8)
    x = torch.randn((4, 300), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    x[1, 7], x[2, 299] = np.nan, np.inf
    y = int4.matmul(x, m)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    w = torch.from_numpy(values[0][:, 299])
    got = y[2].cpu()
    assert torch.isnan(got[w == 0]).all() and (got[w > 0] == np.inf).all() and (got[w < 0] == -np.inf).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pitch,at", [(1000, 0), (1001, 0), (1024, 1), (1024, 8), (1032, 4)])
def test_strides_and_starts(dtype, pitch, at):
    k = 900
    m, values = made(0, 50, k, 2)
    wide = torch.full((6, pitch), np.nan, dtype=dtype, device="cuda")
    x = wide[:, at:at + k]
    x.copy_(torch.randn((6, k), generator=torch.Generator().manual_seed(at)))
    assert torch.equal(int4.matmul(x, m), int4.matmul(x.contiguous(), m))
    check_product(x, m, values, None)


def test_pitch_of_the_output():
    """The C entry point writes rows any distance apart and nothing between them."""
    from lossless_bf16_compression_gb300 import _tensors

    m, _ = made(2, 70, 300, 4)
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    want = int4.matmul(x, m, offsets)
    out = torch.full((5, 90), 5.0, dtype=torch.bfloat16, device="cuda")
    rc = _tensors.fn("zc_int4_matmul")(x.data_ptr(), 300, 0, 5, m.data.data_ptr(), m.scales.data_ptr(), 2, 70, 300, offsets.data_ptr(),
                                       out.data_ptr(), 90, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == zc.ZC_OK
    assert torch.equal(out[:, :70], want) and (out[:, 70:] == 5).all() and (want[4] == 0).all()


def test_streams_and_graphs():
    m, _ = made(6, 200, 1500, 5)
    x = torch.randn((12, 1500), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    offsets = torch.tensor([0, 2, 2, 5, 6, 11, 12], dtype=torch.int32, device="cuda")
    want = int4.matmul(x, m, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = int4.matmul(x, m, offsets, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = int4.matmul(x, m, offsets)
        v = int4.quantize_weight(x).values()
    for o in ([0, 2, 2, 5, 6, 11, 12], [0, 0, 0, 0, 0, 0, 9], [0, 0, 0, 0, 0, 0, 0], [0, 12, 12, 12, 12, 12, 12]):
        offsets.copy_(torch.tensor(o, dtype=torch.int32))
        x.copy_(torch.randn((12, 1500)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, int4.matmul(x, m, offsets)) and torch.equal(v, int4.quantize_weight(x).values())


def test_weights_past_32_bit_offsets():
    """The last of 1000 experts of 2048 x 4608 (4.7 GB of records) and its values (18.9 GB)."""
    groups, n, k = 1000, 2048, 4608
    data = torch.full((groups, n // 16, k // 128, 1024), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones((groups, n // 16, k // 128, 16), dtype=torch.bfloat16, device="cuda")
    one = int4.quantize_weight(torch.randn((n, k), generator=torch.Generator().manual_seed(1)).bfloat16().cuda())
    data[-1], scales[-1] = one.data, one.scales
    m = int4.Matrix(data, scales, n, k)
    offsets = torch.full((groups + 1,), 3, dtype=torch.int32, device="cuda")
    offsets[0], offsets[-1] = 0, 10
    x = torch.randn((10, k), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    y = int4.matmul(x, m, offsets)
    assert (y[:3] == 0).all()
    offsets[:-1] = 0
    z = int4.matmul(x, m, offsets)
    alone = int4.matmul(x, one)
    size = doubles(x.abs().float() @ one.values().abs().t())
    bound = 2 * size * (3 * 128 * 2.0 ** -23 + (2 * k // 128 + 40) * 2.0 ** -24)  # (the cut of the work may differ)
    for a, rows in ((y, slice(3, 10)), (z, slice(0, 10))):
        d = np.abs(doubles(a[rows]) - doubles(alone[rows]))
        assert (d <= bound[rows] + 2 * half_ulp(torch.bfloat16) * (np.abs(doubles(alone[rows])) + bound[rows])).all()
    v = m.values(torch.bfloat16)
    assert torch.equal(v[-1], one.values(torch.bfloat16)) and (v[-2] == 0).all()
    q = int4.quantize_weight(v)
    assert torch.equal(q.data[-1], int4.quantize_weight(v[-1]).data) and (q.data[0] == 0x88).all()


def test_a_product_follows_the_kernels_that_make_its_operands():
    """Rows and weights written just before, by kernels that let the next one start early."""
    from lossless_bf16_compression_gb300 import moe

    w = torch.randn((6, 96, 512), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    xs = [torch.randn((40, 512), generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in range(4)]
    ids = torch.randint(-1, 6, (40, 2), generator=torch.Generator().manual_seed(5)).cuda()

    def step(x):
        rows, plan = moe.dispatch(x, ids, 6)
        return int4.matmul(rows, int4.quantize_weight(w * x[0, 0]), plan.offsets)

    want = []
    for x in xs:
        want.append(step(x))
        torch.cuda.synchronize()
    for _ in range(10):
        for y, x in zip(want, xs):
            assert torch.equal(step(x), y)


def test_two_streams_at_once():
    m, _ = made(8, 300, 1000, 9)
    offsets = torch.tensor([0, 3, 3, 9, 10, 22, 25, 25, 30], dtype=torch.int32, device="cuda")
    xs = [torch.randn((30, 1000), generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in (1, 2)]
    want = [int4.matmul(x, m, offsets) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [int4.matmul(xs[i % 2], m, offsets, stream=streams[i % 2]) for i in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


def test_kernel_times_go_by_their_ids():
    w = torch.ones((64, 256), device="cuda")
    zc.zc_timing_enable(1)
    try:
        zc.zc_timing_collect()
        m = int4.quantize_weight(w)
        m.values()
        int4.matmul(w, m)
        torch.cuda.synchronize()
        seen = [k for k, ms in zc.zc_timing_collect() if ms > 0]
    finally:
        zc.zc_timing_enable(0)
    assert seen == [zc.ZC_KERNEL_INT4_WEIGHT, zc.ZC_KERNEL_INT4_VALUES, zc.ZC_KERNEL_INT4_PRODUCT]


@pytest.mark.parametrize("bad", [[1, 2, 4, 6], [0, 4, 2, 6], [0, 2, 4, 9], [0, -3, 4, 6]])
def test_offsets_that_do_not_fit_are_reported(bad):
    """Every access is clamped to the rows: nothing outside is touched, and the status says so."""
    m, _ = made(3, 40, 256, 6)
    wide = torch.zeros((10, 256), dtype=torch.bfloat16, device="cuda")
    int4.matmul(wide[2:8], m, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert zc.status(reset=True) == zc.ZC_ERR_CORRUPT


def test_rows_and_weights_of_no_size():
    m, _ = made(2, 40, 256, 6)
    y = int4.matmul(torch.zeros((0, 256), device="cuda"), m, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 40) and y.dtype == torch.float32
    with pytest.raises(ValueError):
        int4.quantize_weight(torch.zeros((0, 5), device="cuda"))


def test_refusals():
    m, _ = made(2, 40, 256, 6)
    one, _ = made(0, 40, 256, 6)
    x = torch.zeros((4, 256), device="cuda")
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for args, error in (((x, m), ValueError), ((x, one, offsets), ValueError), ((x[:, :255], m, offsets), ValueError),
                        ((x.double(), m, offsets), TypeError), ((x, m.data, offsets), TypeError), ((x, m, offsets.long()), TypeError),
                        ((x, m, offsets[:2]), ValueError), ((x[0], m, offsets), ValueError), ((x.cpu(), m, offsets), TypeError),
                        ((x, m, offsets, torch.int8), TypeError)):
        with pytest.raises(error):
            int4.matmul(*args)
    with pytest.raises(RuntimeError, match="requires a gradient"):
        int4.matmul(x.clone().requires_grad_(), m, offsets)
    with pytest.raises(TypeError):
        int4.Matrix(m.data.int(), m.scales, 40, 256)
    with pytest.raises(ValueError):
        int4.Matrix(m.data, m.scales, 40, 257)
    with pytest.raises(ValueError):
        int4.Matrix(m.data, m.scales[:, :, :1], 40, 256)
    with pytest.raises(ValueError):
        int4.Matrix(m.data.transpose(1, 2), m.scales, 40, 256)
    with pytest.raises(TypeError):
        one.values(torch.int32)
    one.rows = 64  # exchanged parts are seen by the call
    with pytest.raises(ValueError):
        int4.matmul(x, one)
