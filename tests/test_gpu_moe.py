"""Tokens sorted by expert and back, with their gradients, against 64-bit statements of the same operators.

Tolerances: a sum of k products in fp32 is off by at most k 2^-24 times the sum of the products' magnitudes (one
rounding for each fused multiply-add), and the result is then rounded once to its type.  A dot product over h values
takes at most h + 1 such roundings, whatever its order.  What is only moved or chosen is compared bit for bit.
"""
import numpy as np
import pytest

from gpu_helpers import require_gpu
from moe_oracle import doubles, half_ulp, smallest, sort

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import moe  # noqa: E402

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def routing(tokens, k, experts, seed, dropped=0.1, skew=False):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, k))
    if skew:
        ids[rng.random((tokens, k)) < 0.7] = experts // 2
    gone = rng.random((tokens, k)) < dropped
    ids[gone] = rng.choice([-1, -7, experts, experts + 5], gone.sum())
    return ids


def values(shape, dtype, seed, pitch=0):
    """Seeded values; pitch > 0: rows that far apart in a wider buffer."""
    g = torch.Generator().manual_seed(seed)
    rows, cols = shape
    t = torch.randn((rows, max(pitch, cols)), generator=g).to(dtype).cuda()
    return t[:, :cols]


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(
        a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# (tokens, k, experts, hidden): one token, odd sizes, one expert, more experts than slots, several sort chunks
SHAPES = [(1, 1, 1, 1), (1, 8, 64, 96), (3, 2, 5, 7), (37, 6, 40, 130), (200, 8, 256, 64), (513, 3, 1, 24),
          (1000, 5, 17, 33), (2500, 8, 1024, 8)]


@pytest.mark.parametrize("tokens,k,experts,hidden", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_sort_places_every_slot(tokens, k, experts, hidden, wide):
    ids = routing(tokens, k, experts, tokens + k, skew=tokens > 100)
    want_p, want_o = sort(ids, experts)
    t = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    plan = moe.sort(t, experts)
    assert np.array_equal(plan.position.cpu().numpy(), want_p)
    assert np.array_equal(plan.offsets.cpu().numpy(), want_o)


def test_sort_of_ids_beyond_32_bits():
    ids = torch.tensor([[0, 1 << 32], [-(1 << 32), 3], [(1 << 33) + 1, 2]], device="cuda")
    plan = moe.sort(ids, 4)
    assert plan.offsets.tolist() == [0, 1, 1, 2, 3]
    assert plan.position.tolist() == [[0, 3], [4, 2], [5, 1]]


@pytest.mark.parametrize("tokens", [0, 1, 300])
def test_no_expert_at_all(tokens):
    """Every slot dropped: zeros everywhere, and nothing of the rows (NaN here) comes through."""
    k, experts, hidden = 3, 4, 40
    ids = torch.full((tokens, k), -1, dtype=torch.int32, device="cuda")
    x = torch.full((tokens, hidden), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows, plan = moe.dispatch(x, ids, experts)
    assert plan.offsets.tolist() == [0] * (experts + 1)
    assert rows.shape == (tokens * k, hidden) and not rows.float().abs().sum().item()
    w = torch.full((tokens, k), float("nan"), device="cuda")
    bad = torch.full_like(rows, float("inf"))
    assert not moe.combine(bad, w, plan).float().abs().sum().item()
    d_rows, d_w = moe.combine_grad(x, bad, w, plan)
    assert not d_rows.float().abs().sum().item() and not d_w.abs().sum().item()


def test_many_slots_of_one_call():
    """A sort over many chunks, against the sort of numpy (which the small cases check against the definition)."""
    for tokens, k, experts in ((16384, 8, 64), (70001, 3, 300), (9000, 1, 2)):
        ids = routing(tokens, k, experts, 5, skew=True).reshape(-1)
        key = np.where((ids >= 0) & (ids < experts), ids, experts)
        order = np.argsort(key, kind="stable")
        want = np.empty_like(order)
        want[order] = np.arange(order.size)
        plan = moe.sort(torch.from_numpy(ids.reshape(tokens, k)).to(torch.int32).cuda(), experts)
        assert np.array_equal(plan.position.cpu().numpy().reshape(-1), want)
        assert np.array_equal(plan.offsets.cpu().numpy(), np.searchsorted(key[order], np.arange(experts + 1)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,experts,hidden", SHAPES + [(5, 8, 16, 7168), (300, 2, 8, 2050)])
def test_dispatch_moves_rows(tokens, k, experts, hidden, dtype):
    ids = routing(tokens, k, experts, 3 * tokens)
    x = values((tokens, hidden), dtype, 1, pitch=hidden + (tokens % 3) * 3)
    rows, plan = moe.dispatch(x, torch.from_numpy(ids).to(torch.int32).cuda(), experts)
    want_p, want_o = sort(ids, experts)
    assert np.array_equal(plan.position.cpu().numpy(), want_p) and np.array_equal(plan.offsets.cpu().numpy(), want_o)
    want = torch.zeros((tokens * k, hidden), dtype=dtype)
    xc = x.cpu()
    for t in range(tokens):
        for j in range(k):
            if 0 <= ids[t, j] < experts:
                want[want_p[t, j]] = xc[t]
    assert same_bits(rows.cpu(), want)


def test_dispatch_keeps_every_bit_pattern():
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(32, 2048).cuda()
    ids = torch.arange(32, device="cuda").flip(0)[:, None]
    rows, _ = moe.dispatch(bits.view(torch.bfloat16), ids, 32)
    assert torch.equal(rows.view(torch.int16), bits.flip(0))


def check_sum(got, want, terms, dtype, count):
    bound = count * 2.0 ** -24 * terms + half_ulp(dtype) * (np.abs(want) + count * 2.0 ** -24 * terms) + smallest(dtype)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,experts,hidden", SHAPES + [(5, 8, 16, 7168), (300, 2, 8, 2050), (9, 17, 30, 72)])
def test_combine_adds_rows(tokens, k, experts, hidden, dtype, weighted):
    ids = routing(tokens, k, experts, 7 * tokens, dropped=0.3)
    position, offsets = sort(ids, experts)
    plan = moe.Plan(torch.from_numpy(position).cuda(), torch.from_numpy(offsets).cuda())
    rows = values((tokens * k, hidden), dtype, 2, pitch=hidden + (tokens % 2) * 5)
    rows[offsets[-1]:] = float("nan")  # rows without an expert add nothing
    w = values((tokens, k), torch.float32, 3)
    got = moe.combine(rows, w, plan) if weighted else moe.dispatch_grad(rows, plan)
    r = np.nan_to_num(doubles(rows))[position] * (doubles(w)[..., None] if weighted else 1.0)
    r = np.where((position < offsets[-1])[..., None], r, 0.0)
    assert got.shape == (tokens, hidden) and got.dtype == dtype
    check_sum(doubles(got), r.sum(1), np.abs(r).sum(1), dtype, k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,experts,hidden", SHAPES + [(5, 8, 16, 7168), (300, 2, 8, 2050), (9, 17, 30, 72)])
def test_combine_grad(tokens, k, experts, hidden, dtype):
    ids = routing(tokens, k, experts, 11 * tokens, dropped=0.3)
    position, offsets = sort(ids, experts)
    plan = moe.Plan(torch.from_numpy(position).cuda(), torch.from_numpy(offsets).cuda())
    rows = values((tokens * k, hidden), dtype, 4)
    rows[offsets[-1]:] = float("inf")
    d_out = values((tokens, hidden), dtype, 5, pitch=hidden + (tokens % 2) * 8)
    w = values((tokens, k), torch.float32, 6)
    d_rows, d_w = moe.combine_grad(d_out, rows, w, plan)
    kept = (position < offsets[-1])[..., None]
    d, r = doubles(d_out)[:, None, :], np.where(kept, np.nan_to_num(doubles(rows), posinf=0.0)[position], 0.0)
    want_rows = np.where(kept, d * doubles(w)[..., None], 0.0)
    got_rows = doubles(d_rows)[position]
    check_sum(got_rows, want_rows, np.abs(want_rows), dtype, 1)
    prod = d * r
    check_sum(doubles(d_w), prod.sum(2), np.abs(prod).sum(2), torch.float32, hidden + 1)


@pytest.mark.parametrize("tokens,k,hidden", [(2100, 1, 24), (2101, 2, 36), (2103, 3, 7), (2049, 4, 40), (2050, 7, 10)])
def test_many_tokens_of_few_slots(tokens, k, hidden):
    """Token counts at which a thread takes several tokens, not a multiple of them."""
    ids = routing(tokens, k, 11, tokens)
    position, offsets = sort(ids, 11)
    plan = moe.Plan(torch.from_numpy(position).cuda(), torch.from_numpy(offsets).cuda())
    rows, w = values((tokens * k, hidden), torch.bfloat16, 1), values((tokens, k), torch.float32, 2)
    r = np.where((position < offsets[-1])[..., None], doubles(rows)[position], 0.0)
    check_sum(doubles(moe.dispatch_grad(rows, plan)), r.sum(1), np.abs(r).sum(1), torch.bfloat16, k)
    r = r * doubles(w)[..., None]
    check_sum(doubles(moe.combine(rows, w, plan)), r.sum(1), np.abs(r).sum(1), torch.bfloat16, k)


def test_gradients_against_differences():
    """combine and dispatch are linear in rows and in weights: central differences of the loss <out, g>, in fp32.

    The loss is a sum of fp32 outputs weighted in 64 bits; each output carries at most k 2^-24 of its terms, so a
    difference over 2 h is off by at most that over h (h = 1/8, where x + h and x - h are rounded as well)."""
    tokens, k, experts, hidden, h = 6, 3, 4, 9, 0.125
    ids = torch.from_numpy(routing(tokens, k, experts, 9, dropped=0.25)).cuda()
    x = values((tokens, hidden), torch.float32, 1)
    w, g = values((tokens, k), torch.float32, 2), values((tokens, hidden), torch.float32, 3)
    rows, plan = moe.dispatch(x, ids, experts)
    scale = np.abs(doubles(rows)).max() + 1
    bound = (k + 2) * 2.0 ** -23 * scale * (np.abs(doubles(w)).max() + 1) * np.abs(doubles(g)).sum() * k / h

    def loss(x_, w_):
        r, p = moe.dispatch(x_, ids, experts)
        return float((doubles(moe.combine(r, w_, p)) * doubles(g)).sum())

    d_rows, d_w = moe.combine_grad(g, rows, w, plan)
    dx = moe.dispatch_grad(d_rows, plan)
    for grad, t, f in ((dx, x, lambda t_: loss(t_, w)), (d_w, w, lambda t_: loss(x, t_))):
        for i in range(t.shape[0]):
            for j in range(t.shape[1]):
                up, down = t.clone(), t.clone()
                up[i, j] += h
                down[i, j] -= h
                assert abs((f(up) - f(down)) / (2 * h) - grad[i, j].item()) <= bound


def test_rows_past_32_bit_offsets():
    """Sorted rows whose bytes pass 2^32 (and whose values pass 2^31)."""
    tokens, k, experts, hidden = 40000, 8, 4, 7168
    x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = (torch.arange(tokens, device="cuda") % 251).to(torch.bfloat16)
    x[:, -1] = (torch.arange(tokens, device="cuda") % 127).to(torch.bfloat16)
    ids = ((torch.arange(tokens, device="cuda")[:, None] + torch.arange(k, device="cuda")) % experts).to(torch.int32)
    rows, plan = moe.dispatch(x, ids, experts)
    at = plan.position.long()
    assert rows.numel() > 1 << 31
    assert torch.equal(rows[:, 0][at], x[:, :1].expand(-1, k)) and torch.equal(rows[:, -1][at], x[:, -1:].expand(-1, k))
    out = moe.dispatch_grad(rows, plan)
    assert torch.equal(out[:, 0], (x[:, 0].float() * k).to(torch.bfloat16))
    assert torch.equal(out[:, -1], (x[:, -1].float() * k).to(torch.bfloat16))


def test_same_bits_every_time():
    ids = torch.from_numpy(routing(777, 6, 20, 1)).cuda()
    x, w = values((777, 258), torch.bfloat16, 1), values((777, 6), torch.float32, 2)

    def step():
        rows, plan = moe.dispatch(x, ids, 20)
        out = moe.combine(rows, w, plan)
        d_rows, d_w = moe.combine_grad(out, rows, w, plan)
        return rows, out, d_rows, d_w, moe.dispatch_grad(d_rows, plan)

    first = step()
    for _ in range(3):
        assert all(same_bits(a, b) for a, b in zip(first, step()))


def test_strided_ids_weights_and_columns():
    """Inputs that are not laid out in rows are taken as they are read."""
    ids = torch.from_numpy(routing(50, 8, 6, 2)).cuda()[:, ::2]
    x = values((64, 50), torch.float16, 1).t()  # [50, 64], columns contiguous
    w = values((4, 50), torch.float32, 2).t()
    rows, plan = moe.dispatch(x, ids, 6)
    rows2, plan2 = moe.dispatch(x.contiguous(), ids.contiguous(), 6)
    assert same_bits(rows, rows2) and same_bits(plan.position, plan2.position)
    assert same_bits(moe.combine(rows, w, plan), moe.combine(rows, w.contiguous(), plan))


def test_on_another_stream():
    ids = torch.from_numpy(routing(333, 4, 9, 3)).cuda()
    x, w = values((333, 128), torch.bfloat16, 1), values((333, 4), torch.float32, 2)
    rows, plan = moe.dispatch(x, ids, 9)
    out = moe.combine(rows, w, plan)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rows2, plan2 = moe.dispatch(x, ids, 9, stream=side)
    out2 = moe.combine(rows2, w, plan2, stream=side)
    side.synchronize()
    assert same_bits(rows, rows2) and same_bits(out, out2)


def test_captured_in_a_graph():
    """One capture, replayed on another routing of the same shape."""
    shape, experts = (700, 6), 12
    ids = torch.from_numpy(routing(*shape, experts, 3)).to(torch.int32).cuda()
    x, w = values((700, 64), torch.bfloat16, 1), values(shape, torch.float32, 2)

    def step():
        rows, plan = moe.dispatch(x, ids, experts)
        return rows, plan.position, moe.combine(rows, w, plan)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    ids.copy_(torch.from_numpy(routing(*shape, experts, 4)))
    g.replay()
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, step()))
    del g


def test_position_out_of_range_is_skipped_and_reported():
    plan = moe.Plan(torch.tensor([[0, 99], [-3, 1]], dtype=torch.int32, device="cuda"),
                    torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    rows = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    out = moe.combine(rows, w, plan)
    assert zc.status(reset=True) == zc.ZC_ERR_CORRUPT
    assert torch.equal(out, torch.ones_like(out))
    moe.combine_grad(out, rows, w, plan)
    assert zc.status(reset=True) == zc.ZC_ERR_CORRUPT


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    rows, plan = moe.dispatch(x, ids, 3)
    w = torch.zeros((4, 2), device="cuda")
    for call in (lambda: moe.dispatch(x.cpu(), ids, 3), lambda: moe.dispatch(x.double(), ids, 3),
                 lambda: moe.dispatch(x, ids.float(), 3), lambda: moe.combine(rows, w.half(), plan),
                 lambda: moe.combine_grad(x.float(), rows, w, plan), lambda: moe.sort(ids.tolist(), 3)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: moe.dispatch(x[:3], ids, 3), lambda: moe.dispatch(x, ids, 0), lambda: moe.dispatch(x, ids, 1025),
                 lambda: moe.dispatch(x, ids[:, :0], 3), lambda: moe.dispatch(x[:, :0], ids, 3),
                 lambda: moe.dispatch(x, ids.reshape(-1), 3), lambda: moe.combine(rows[:5], w, plan),
                 lambda: moe.combine(rows, w[:, :1], plan), lambda: moe.combine_grad(x[:, :4], rows, w, plan),
                 lambda: moe.sort(ids.expand(65, 4, 2).reshape(4, 130), 3)):
        with pytest.raises(ValueError):
            call()
