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


def two(s):
    """2^s in 64 bits, by the bits."""
    return ((s + 1023) << 52).view(torch.float64)


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


# ------------------------------------------------------------------ the products' bounded waits


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def stalled_matmul(a, b, offsets, cta, wait_us):
    from lossless_bf16_compression_gb300 import _tensors

    groups, n = b.data.shape[:2]
    out = torch.zeros((a.rows, n), device="cuda")
    need = _tensors.fn("zc_fp8_matmul_workspace")(a.rows, groups, n, a.cols)
    scratch = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    rc = _tensors.fn("zc_fp8_matmul_stall_test")(
        a.data.data_ptr(), a.scales.data_ptr(), 0, a.rows, b.data.data_ptr(), b.scales.data_ptr(), 0, groups, n, a.cols,
        offsets.data_ptr(), out.data_ptr(), n, 2, scratch.data_ptr() if need else 0,
        torch.cuda.current_stream().cuda_stream, cta, wait_us)
    assert rc == zc.ZC_OK
    return out, need


def stalled_weight_grad(dy, x, cta, wait_us):
    from lossless_bf16_compression_gb300 import _tensors

    groups = x.offsets.numel() - 1
    out = torch.zeros((groups, dy.rows, x.rows), device="cuda")
    rc = _tensors.fn("zc_fp8_weight_grad_stall_test")(
        dy.data.data_ptr(), dy.scales.data_ptr(), 0, x.data.data_ptr(), x.scales.data_ptr(), 0, x.data.shape[1] // 128,
        groups, dy.rows, x.rows, x.offsets.data_ptr(), out.data_ptr(), 2, torch.cuda.current_stream().cuda_stream, cta,
        wait_us)
    assert rc == zc.ZC_OK
    return out


# single CTAs, pairs (256 x 256 tiles: 16 rounds of them at 4096 x 4096), blocks shared out (a workspace)
@pytest.mark.parametrize("counts,n,k,shared", [((300,), 200, 640, False), ((4096,), 4096, 700, False),
                                               ((3, 0, 5), 1000, 7168, True)])
@pytest.mark.parametrize("cta", [0, 1])
def test_a_product_whose_loads_never_come_gives_up(counts, n, k, shared, cta):
    """The waits run out, the status says so, and the call after it is whole."""
    at = starts(counts)
    a = fp8.quantize(values((int(at[-1]), k), torch.bfloat16, 1))
    b, _ = fp8.quantize_weight(values((len(counts), n, k), torch.bfloat16, 2), transposed=False)
    want = fp8.matmul(a, b, at, torch.float32)
    for _ in range(2):
        _, need = stalled_matmul(a, b, at, cta, 20000)
        assert zc.status(reset=True) == zc.ZC_ERR_TIMEOUT and (need > 0) == shared
        assert same_bits(fp8.matmul(a, b, at, torch.float32), want)
        assert same_bits(stalled_matmul(a, b, at, -1, 200000)[0], want)
        assert zc.status(reset=True) == zc.ZC_OK


@pytest.mark.parametrize("counts,n,k", [((100, 0, 30), 200, 130), ((600,) * 8, 2048, 1024)])
@pytest.mark.parametrize("cta", [0, 1])
def test_a_weight_gradient_whose_loads_never_come_gives_up(counts, n, k, cta):
    at = starts(counts)
    dy = fp8.quantize_columns(values((int(at[-1]), n), torch.bfloat16, 1), at)
    x = fp8.quantize_columns(values((int(at[-1]), k), torch.bfloat16, 2), at)
    want = fp8.weight_grad(dy, x, torch.float32)
    for _ in range(2):
        stalled_weight_grad(dy, x, cta, 20000)
        assert zc.status(reset=True) == zc.ZC_ERR_TIMEOUT
        assert same_bits(fp8.weight_grad(dy, x, torch.float32), want)
        assert same_bits(stalled_weight_grad(dy, x, -1, 200000), want)
        assert zc.status(reset=True) == zc.ZC_OK


def test_a_sum_longer_than_the_limit_of_a_wait_is_not_given_up():
    """65,536 blocks in one tile take about 20 ms, ten times the limit given here for any other wait.  Ones far apart,
    so that the sum is exact."""
    rows = 1 << 23
    dy, x = torch.zeros((rows, 1), dtype=torch.bfloat16, device="cuda"), torch.ones((rows, 3), dtype=torch.bfloat16, device="cuda")
    dy[::65536] = 1
    got = stalled_weight_grad(fp8.quantize_columns(dy), fp8.quantize_columns(x), -1, 2000)
    assert zc.status(reset=True) == zc.ZC_OK
    assert got.flatten().tolist() == [128.0] * 3


# ------------------------------------------------------------------ every number of experts

SORTS = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
from lossless_bf16_compression_gb300 import moe
experts, wide = int(sys.argv[2]), sys.argv[3] == "wide"
for slots, k in ((2, 2), (3000, 3)):
    ids = (torch.arange(slots, device="cuda") * 7 % (experts + 1)).view(-1, k)
    key = ids.reshape(-1)
    order = torch.argsort(key, stable=True)
    want = torch.empty_like(order)
    want[order] = torch.arange(slots, device="cuda")
    starts = torch.searchsorted(key[order], torch.arange(experts + 1, device="cuda"))
    x = torch.arange(slots // k * 4, device="cuda").view(-1, 4).float()
    for plan in (moe.sort(ids if wide else ids.int(), experts), moe.dispatch(x, ids if wide else ids.int(), experts)[1]):
        assert torch.equal(plan.position.reshape(-1).long(), want) and torch.equal(plan.offsets.long(), starts)
print("ok")
"""


@pytest.mark.parametrize("experts,ids", [(765, "int"), (766, "int"), (767, "int"), (767, "wide"), (768, "wide"), (1023, "int")])
def test_sort_of_as_many_experts_as_the_first_call_asks_for(experts, ids):
    """In a process of its own: what an earlier call asked of the device does not help this one."""
    r = subprocess.run([sys.executable, "-c", SORTS, ROOT, str(experts), ids], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr


def test_sorts_of_two_threads():
    """One thread's call does not take back what the other's needs."""
    import threading

    from lossless_bf16_compression_gb300 import _tensors

    fn, calls, codes = _tensors.fn("zc_moe_sort"), 300, []
    ids = torch.zeros(2000, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def work(experts):
        position, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (2000, experts + 1))
        scratch = torch.empty(_tensors.fn("zc_moe_sort_workspace")(2000, experts), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        codes.extend(fn(ids.data_ptr(), 4, 1000, 2, experts, position.data_ptr(), offsets.data_ptr(), scratch.data_ptr(),
                        stream.cuda_stream) for _ in range(calls))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(e,)) for e in (1024, 800, 900)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [zc.ZC_OK] * (3 * calls)


# ------------------------------------------------------------------ matrices of a program's own making


def dequantized(m):
    s = two(m.scales.long() - 127).transpose(0, 1).reshape(m.rows, -1)[:, : m.data.shape[1] // 128]
    return m.values().double() * s.repeat_interleave(128, 1)[:, : m.cols]


def test_weight_grad_of_rows_that_end_inside_a_block():
    """Blocks along the rows of two matrices, with starts of the program's own: the last block counts though it is not full.
    Sums of 300 terms in fp32 (tolerance as for the products' tests: 300 2^-23 of the terms' magnitudes)."""
    a, b = fp8.quantize(values((5, 300), torch.float32, 1)), fp8.quantize(values((7, 300), torch.float32, 2))
    starts_of = torch.tensor([0, 2, 2, 3], dtype=torch.int32, device="cuda")
    dy, x = (fp8.Matrix(m.data, m.scales, 300, offsets=starts_of) for m in (a, b))
    got = fp8.weight_grad(dy, x, torch.float32).double()
    assert zc.status(reset=True) == zc.ZC_OK
    va, vb = dequantized(a), dequantized(b)
    for g, (lo, hi) in enumerate(((0, 256), (256, 256), (256, 300))):
        p, q = va[:, lo:hi], vb[:, lo:hi]
        assert ((got[g] - p @ q.T).abs() <= 300 * 2.0 ** -23 * (p.abs() @ q.abs().T)).all()


def test_exchanged_tensors_are_refused():
    """A Matrix whose tensors were exchanged after it was made: no call reads past them."""
    at = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")

    def matrix(rows, cols):
        m = fp8.quantize(values((rows, cols), torch.float32, rows))
        return fp8.Matrix(m.data, m.scales, cols, offsets=at)

    good = matrix(40, 300)
    for change in (lambda m: setattr(m, "scales", m.scales[:, :39]), lambda m: setattr(m, "scales", m.scales[:0]),
                   lambda m: setattr(m, "scales", m.scales.expand(2, 40, 4)[:, ::2]),
                   lambda m: setattr(m, "data", matrix(41, 300).data), lambda m: setattr(m, "data", m.data[:, :256]),
                   lambda m: setattr(m, "data", matrix(40, 500).data[:, :384]), lambda m: setattr(m, "data", m.data[0]),
                   lambda m: setattr(m, "cols", 385), lambda m: setattr(m, "cols", 0), lambda m: setattr(m, "cols", -5)):
        bad = matrix(40, 300)
        change(bad)
        for call in (lambda: fp8.matmul(good, bad), lambda: fp8.matmul(bad, good), lambda: fp8.weight_grad(good, bad),
                     lambda: fp8.weight_grad(bad, good)):
            with pytest.raises(ValueError):
                call()
    bad = matrix(40, 300)
    bad.scales = torch.zeros((1, 40, 8), dtype=torch.uint8, device="cuda")[:, :, ::2]
    with pytest.raises(ValueError):
        bad.scale_values()
    bad.scales = torch.zeros(7, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        bad.scale_values()
    for offsets in ([0, 1], at.long(), at.tolist()):
        with pytest.raises(TypeError):
            fp8.Matrix(good.data, good.scales, 300, offsets=offsets)
    assert fp8.matmul(good, good).shape == (40, 40) and fp8.weight_grad(good, good).shape == (2, 40, 40)


# ------------------------------------------------------------------ tensors that require a gradient


def test_a_gradient_is_not_lost_unseen():
    """A result would have no history, so an input that requires a gradient is refused where gradients are recorded, and
    taken where they are not: under no_grad, detached, in a function's forward."""
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = values((4, 256), torch.float32, 1).requires_grad_()
    w = values((4, 2), torch.float32, 2).requires_grad_()
    rows, plan = moe.dispatch(x.detach(), ids, 3)
    calls = [lambda t: moe.dispatch(t(x), ids, 3), lambda t: moe.combine(rows, t(w), plan),
             lambda t: moe.combine(t(rows.clone().requires_grad_()), w.detach(), plan),
             lambda t: moe.combine_grad(t(x), rows, w.detach(), plan), lambda t: moe.dispatch_grad(t(rows.clone().requires_grad_()), plan),
             lambda t: fp8.quantize(t(x)), lambda t: fp8.quantize_columns(t(x)), lambda t: fp8.quantize_weight(t(x))]
    for call in calls:
        with pytest.raises(RuntimeError, match="requires a gradient"):
            call(lambda v: v)
        call(lambda v: v.detach())
        with torch.no_grad():
            call(lambda v: v)
        with torch.inference_mode():
            call(lambda v: v)

    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            r, ctx.plan = moe.dispatch(t, ids, 3)
            return r

        @staticmethod
        def backward(ctx, d):
            return moe.dispatch_grad(d, ctx.plan)

    Dispatch.apply(x).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


# ------------------------------------------------------------------ kernel timing


def test_every_kernel_is_timed():
    """zc_timing_enable brackets every kernel that the library launches, the experts' among them."""
    x, w = values((1000, 256), torch.bfloat16, 1), values((1000, 4), torch.float32, 2)
    ids = routing(1000, 4, 9, 3)
    few = starts((3, 0, 5))
    a = fp8.quantize(values((8, 7168), torch.bfloat16, 4))

    def step():
        """The calls, and the ids of the kernels that each launches."""
        s, d, c, cg = zc.ZC_KERNEL_MOE_SORT, zc.ZC_KERNEL_MOE_DISPATCH, zc.ZC_KERNEL_MOE_COMBINE, zc.ZC_KERNEL_MOE_COMBINE_GRAD
        q, col, wt, sc, p = (zc.ZC_KERNEL_FP8_ROWS, zc.ZC_KERNEL_FP8_COLUMNS, zc.ZC_KERNEL_FP8_WEIGHT, zc.ZC_KERNEL_FP8_SCALES,
                             zc.ZC_KERNEL_FP8_PRODUCT)
        out, kernels = [], []

        def take(values_, *names):
            out.extend(v for v in values_ if isinstance(v, torch.Tensor))
            kernels.extend(names)
            return values_

        rows, plan = take(moe.dispatch(x, ids, 9), s, s, d)
        take([rows, *plan])
        take(moe.dispatch(x[:7], ids[:7], 9), d)
        take(moe.sort(ids[:7], 9), s)
        back = take([moe.combine(rows, w, plan)], c)[0]
        take(moe.combine_grad(back, rows, w, plan), cg)
        take([moe.dispatch_grad(rows, plan)], c)
        m = take([fp8.quantize(rows)], q)[0]
        take([m.data, m.scales, m.scale_values()], sc)
        b, b_t = take(fp8.quantize_weight(values((9, 96, 256), torch.bfloat16, 5)), wt)
        y = take([fp8.matmul(m, b, plan.offsets)], p)[0]
        dy, xc = take([fp8.quantize_columns(y, plan.offsets), fp8.quantize_columns(rows, plan.offsets)], col, col)
        take([fp8.weight_grad(dy, xc), b_t.data], p)
        v = take(fp8.quantize_weight(values((2, 1000, 7168), torch.bfloat16, 6), transposed=False), wt)[0]
        v3 = fp8.Matrix(torch.cat([v.data, v.data[:1]]), torch.cat([v.scales, v.scales[:1]]), 7168)
        take([fp8.matmul(a, v3, few)], p, p)  # shared out: its workspace is cleared first
        return out, kernels

    want, _ = step()
    zc.zc_timing_enable(1)
    zc.zc_timing_collect()
    try:
        got, kernels = step()
        records = zc.zc_timing_collect()
    finally:
        zc.zc_timing_enable(0)
    assert [k for k, _ in records] == kernels
    assert all(0 < ms < 1000 for _, ms in records)
    assert all(same_bits(p, q) for p, q in zip(want, got)) and len(want) == len(got)
    step()
    assert zc.zc_timing_collect() == []


# ------------------------------------------------------------------ sizes at which a call takes another kernel


def check_rows(x, fmt):
    """quantize(x) against the definition in 64 bits, on the GPU: each scale the smallest power of two that brings the
    block's largest value into the format, each value one of the two neighbours on the format's grid, the nearer one, at
    a tie the one with the even last bit."""
    from moe_oracle import grid_values

    top = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
    grid = torch.from_numpy(grid_values(fmt)).cuda()
    m = fp8.quantize(x, fmt)
    r, c = x.shape
    blocks = -(-c // 128)
    for a in range(0, r, 4096):
        wide = torch.zeros((min(4096, r - a), blocks * 128), dtype=torch.float64, device="cuda")
        wide[:, :c] = x[a:a + 4096].double()
        wide = wide.view(wide.shape[0], blocks, 128)
        amax = wide.abs().amax(2)
        words = m.scales[:, a:a + 4096].permute(1, 0, 2).reshape(wide.shape[0], -1).long() - 127
        assert not words[:, blocks:].any()
        s = words[:, :blocks]
        scale = two(s)
        zero = amax == 0
        assert (amax <= top * scale).all() and ((amax > top * scale / 2) | (s == -127) | zero).all() and not s[zero].any()
        v = wide / scale[..., None]
        got = m.data[a:a + 4096].view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double().view(v.shape)
        hi = torch.searchsorted(grid, v.abs().contiguous()).clamp(max=grid.numel() - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - v.abs(), v.abs() - grid[lo]
        want = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
        assert torch.equal(got, torch.copysign(want, v))


# from 2048 CTAs of four rows a warp on, a warp takes four rows (two where rows start anywhere): sizes on either side,
# a last warp and a last CTA that are not full, and a last word of scales that is not
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(32768, 300), (32749, 296), (32751, 301), (8195, 2048), (8197, 1999), (6000, 2504)])
def test_quantize_many_rows(rows, cols, dtype, fmt):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda").mul_(1.5).sub_(3).exp_()
    x *= torch.where(torch.rand((rows, cols), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x[torch.rand((rows, cols), generator=g, device="cuda") < 0.01] = 0
    x[rows // 2, :] = 0
    check_rows(x.to(dtype), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,k,hidden,shift", [(600, 3, 7001, 0), (600, 3, 4600, 3), (2100, 2, 2055, 1), (2100, 3, 7168, 0),
                                                   (2049, 5, 4099, 1), (2050, 1, 8200, 0)])
def test_rows_of_several_parts(tokens, k, hidden, shift, dtype):
    """Rows of more than one CTA's or one warp's vectors, aligned or starting anywhere, in calls of more than 1024 slots and
    on either side of 2048 tokens.  Sums: k products of fp32, or hidden of them, and a rounding (test_gpu_moe.py)."""
    experts = 11
    wide = values((tokens, hidden + shift), dtype, 1)
    x, d_out = wide[:, shift:], values((tokens, hidden + 2 * shift), dtype, 2)[:, shift:shift + hidden]
    ids, w = routing(tokens, k, experts, 3, dropped=0.2), values((tokens, k), torch.float32, 4)
    rows, plan = moe.dispatch(x, ids, experts)
    at, kept = plan.position.long(), (ids >= 0)[..., None]
    assert same_bits(rows[at], torch.where(kept, x[:, None, :], torch.zeros((), dtype=dtype, device="cuda")))
    assert plan.offsets[-1].item() == int(kept.sum())

    eps, last = 2.0 ** -24, {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    sources = values((tokens * k, hidden + shift), dtype, 5)[:, shift:]
    r = torch.where(kept, sources.double()[at], 0.0)

    def close(got, want, size, count, rounding):
        err = count * eps * size
        assert ((got.double() - want).abs() <= err + rounding * (want.abs() + err)).all()

    p = r * w.double()[..., None]
    close(moe.combine(sources, w, plan), p.sum(1), p.abs().sum(1), k, last)
    close(moe.dispatch_grad(sources, plan), r.sum(1), r.abs().sum(1), k, last)
    d_rows, d_w = moe.combine_grad(d_out, sources, w, plan)
    want = torch.where(kept, d_out.double()[:, None, :] * w.double()[..., None], 0.0)
    close(d_rows[at], want, want.abs(), 1, last)
    p = r * d_out.double()[:, None, :]
    close(d_w, p.sum(2), p.abs().sum(2), hidden + 1, eps)


@pytest.mark.parametrize("counts,n,k", [((1,) * 40 + (1500,) + (0,) * 10, 260, 300), ((2, 900) + (0,) * 60, 140, 6000),
                                        ((0,) * 5 + (3000,) + (1,) * 7, 700, 520), ((1000,) + (0,) * 1000, 130, 129)])
def test_products_of_a_group_with_most_of_the_rows(counts, n, k):
    """Tiles are cut for the average group: one group of many times as many rows, products and weight gradient (tolerances
    as in test_gpu_fp8.py: the number of terms times 2^-23 of their magnitudes)."""
    at = starts(counts)
    rows, e = int(at[-1]), len(counts)
    a, (b, _) = fp8.quantize(values((rows, k), torch.bfloat16, 1)), fp8.quantize_weight(values((e, n, k), torch.bfloat16, 2))
    got, av = fp8.matmul(a, b, at, torch.float32).double(), dequantized(a)
    dy, x = fp8.quantize_columns(values((rows, n), torch.bfloat16, 3), at), fp8.quantize_columns(values((rows, k), torch.bfloat16, 4), at)
    dw, yv, xv, blocks = fp8.weight_grad(dy, x, torch.float32).double(), dequantized(dy), dequantized(x), dy.offsets.tolist()
    assert zc.status(reset=True) == zc.ZC_OK
    for g in range(e):
        if counts[g] == 0:
            assert not dw[g].any()
            continue
        s = slice(at[g].item(), at[g + 1].item())
        bv = dequantized(fp8.Matrix(b.data[g], b.scales[g], k))
        assert ((got[s] - av[s] @ bv.T).abs() <= k * 2.0 ** -23 * (av[s].abs() @ bv.abs().T)).all()
        s = slice(128 * blocks[g], 128 * blocks[g + 1])
        p, q = yv[:, s], xv[:, s]
        assert ((dw[g] - p @ q.T).abs() <= p.shape[1] * 2.0 ** -23 * (p.abs() @ q.abs().T)).all()


# ------------------------------------------------------------------ NaN, infinities, subnormals, the largest values


def patterns(dtype):
    """[512, 128]: every pattern of a 16-bit type, or 65,536 of 32 bits over all exponents and both signs, shuffled."""
    g = torch.Generator().manual_seed(3)
    bits = torch.arange(1 << 16, dtype=torch.int64)
    if dtype == torch.float32:
        low = torch.randint(0, 1 << 16, (1 << 16,), generator=g)
        low[::5] = 0  # (so that infinities are among them)
        bits = bits << 16 | low
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    else:
        bits = torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16)
    return bits[torch.randperm(1 << 16, generator=g)].view(dtype).view(512, 128)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("ordered", [False, True])
def test_every_quantization_of_every_value(dtype, fmt, ordered):
    """Rows, columns and weights against the 64-bit statements, values and scales for equality: blocks of values of all
    magnitudes with NaN and infinities among them, and (ordered) blocks of neighbours, finite or not as a whole."""
    from moe_oracle import doubles, quantize, quantize_blocks, quantize_columns, unpack_scales

    x = patterns(dtype)
    if ordered:
        key = x.view(torch.int16 if dtype != torch.float32 else torch.int32).reshape(-1)
        x = key.sort().values.view(dtype).view(512, 128)
    x = x.cuda()

    def check(m, v, s):
        got = m.values().float().cpu().numpy().astype(np.float64)
        assert np.array_equal(got, v, equal_nan=True) and np.array_equal(np.signbit(got[v == 0]), np.signbit(v[v == 0]))
        assert np.array_equal(unpack_scales(m.scales.cpu().numpy(), s.shape[1]), s)

    check(fp8.quantize(x, fmt), *quantize(doubles(x), fmt))
    turned = x.t().contiguous()  # a column of 128 x 512 is a row of x
    check(fp8.quantize_columns(turned, None, fmt), *quantize_columns(doubles(turned), np.array([0, 128]), fmt)[:2])
    w = x.reshape(4, 128, 128)
    m, t = fp8.quantize_weight(w, fmt)
    v, s = quantize_blocks(doubles(w).reshape(1, 4, 128 * 128), fmt)
    for e in range(4):
        ve, se = v[0, e].reshape(128, 128), np.full((128, 1), s[0, e])
        check(fp8.Matrix(m.data[e], m.scales[e], 128, fmt), ve, se)
        check(fp8.Matrix(t.data[e], t.scales[e], 128, fmt), ve.T, se)

