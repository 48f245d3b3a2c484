"""A router's choice of experts, its balance loss and their gradients, against 64-bit statements of the same operators.

Tolerances, in units of e = 2^-24 (half a step of fp32): an exponential is off by at most 4 (2 steps, CUDA's bound) and by
its argument's rounding, |x - m|; a sum of positive terms by 1 for each addition on the longest way through it (N terms of
a lane and 5 exchanges, N at most 32); divisions and products by 1 each.  A score's relative error is therefore below
D + 60 units, D the row's spread of logits (D + 4 for the score, D + 4 + 37 + 1 for the sum, the rest spare), and a
gradient w (g - sum g w) is off by at most w (|g| + sum |g| w) (2 D + 180) units, with up to 64 slots in the sum.  Results of
16 bits are then rounded once.  Ids and counts have to be equal.
"""
import numpy as np
import pytest

import router_oracle as oracle
from gpu_helpers import require_gpu
from moe_oracle import doubles, half_ulp, smallest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import moe  # noqa: E402

E = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
KINDS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]
# (tokens, experts, k): one of all, odd sizes, every number of values a lane holds, all experts, many slots
SHAPES = [(1, 1, 1), (3, 5, 2), (130, 40, 6), (33, 64, 8), (17, 65, 3), (64, 128, 8), (21, 200, 8), (40, 256, 8), (9, 257, 33),
          (5, 1024, 64), (7, 31, 31), (2, 64, 64), (1000, 8, 2)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _status():
    zc.status(reset=True)
    yield
    assert zc.status(reset=True) == zc.ZC_OK


def make(tokens, experts, dtype, seed, masked=0.0, padded=0.0, pitch=0, at=0):
    """Seeded logits, with ties in 16 bits; pitch > 0: rows in a wider buffer, starting at column `at`."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, experts), generator=g) * 2
    if masked:
        x[torch.rand((tokens, experts), generator=g) < masked] = -np.inf
    if padded:
        x[torch.rand(tokens, generator=g) < padded] = -np.inf
    x = x.to(dtype)
    if pitch:
        wide = torch.full((tokens, pitch), 77.0, dtype=dtype)
        wide[:, at:at + experts] = x
        return wide.cuda()[:, at:at + experts]
    return x.cuda()


def spread(x):
    """The largest distance between finite logits of a row."""
    finite = np.where(np.isfinite(x), x, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            s = np.nanmax(finite, 1) - np.nanmin(finite, 1)
    return np.nan_to_num(s)[:, None]


def check_route(x, k, score, normalize, scale=1.0):
    w, ids = moe.route(x, k, score, normalize, scale)
    assert w.dtype == torch.float32 and ids.dtype == torch.int32 and w.shape == ids.shape == (x.shape[0], k)
    v = doubles(x)
    want = oracle.choose(v, k)
    assert np.array_equal(ids.cpu().numpy(), want)
    ww = oracle.weights(v, want, score, normalize, scale)
    assert (np.abs(doubles(w) - ww) <= (spread(v) + 60) * E * np.abs(ww) + 2.0 ** -126).all()
    return w, ids


def grad_bound(x, dw, ids, score, normalize, scale=1.0):
    """The largest error of route_grad before rounding: w (|g| + sum |g| w) (2 D + 180) units at every expert."""
    w = np.abs(oracle.weights(x, ids, score, normalize))
    g = np.where(ids >= 0, np.abs(scale * dw), 0)
    total = (g * w).sum(1, keepdims=True)
    out = oracle.probabilities(x, "softmax") * total if (score, normalize) == ("softmax", False) else np.zeros(x.shape)
    for t in range(len(x)):
        kept = (ids[t] >= 0) & (ids[t] < x.shape[1])
        np.add.at(out[t], ids[t][kept], (w[t] * (g[t] + total[t]))[kept])
    return out * (2 * spread(x) + 180) * E


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("tokens,experts,k", SHAPES)
def test_route_and_its_gradient(tokens, experts, k, score, normalize, dtype):
    x = make(tokens, experts, dtype, tokens + experts, masked=0.2 if experts > 30 else 0.0, padded=0.1)
    w, ids = check_route(x, k, score, normalize, 2.5)
    dw = torch.randn((tokens, k), generator=torch.Generator().manual_seed(k)).cuda()
    d = moe.route_grad(dw, x, ids, score, normalize, 2.5)
    assert d.dtype == dtype and d.shape == x.shape
    v, i = doubles(x), ids.cpu().numpy()
    want = oracle.route_grad(doubles(dw), v, i, score, normalize, 2.5)
    bound = grad_bound(v, doubles(dw), i, score, normalize, 2.5)
    assert (np.abs(doubles(d) - want) <= bound + half_ulp(dtype) * (np.abs(want) + bound) + smallest(dtype)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", SHAPES + [(0, 7, 2), (700, 16, 4), (5000, 40, 6)])
def test_balance_and_its_gradient(tokens, experts, k, score, dtype):
    x = make(tokens, experts, dtype, tokens + experts + 1, masked=0.2 if experts > 30 else 0.0, padded=0.15)
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, experts + 1, (tokens, k)).astype(np.int32)  # some of no expert
    b = moe.balance(x, torch.from_numpy(ids).cuda(), score)
    v = doubles(x)
    loss, counts, slope = oracle.balance(v, ids, score)
    assert b.counts.dtype == torch.int32 and np.array_equal(b.counts.cpu().numpy(), counts)
    assert (np.abs(doubles(b.slope) - slope) <= E * slope).all()
    # a sum over tokens: at most tokens / 16 + 200 additions one after the other
    top = spread(v).max() if tokens else 0
    assert b.loss.shape == () and abs(float(b.loss) - loss) <= (top + 260 + tokens / 16) * E * loss
    d_loss = torch.tensor(0.7, device="cuda")
    d = moe.balance_grad(d_loss, x, b, score)
    want = oracle.balance_grad(float(d_loss), v, doubles(b.slope), score)
    p = oracle.probabilities(v, score)
    bound = float(d_loss) * p * (doubles(b.slope) + (p * doubles(b.slope)).sum(1, keepdims=True)) * (2 * spread(v) + 180) * E
    assert d.dtype == dtype and d.shape == x.shape
    assert (np.abs(doubles(d) - want) <= bound + half_ulp(dtype) * (np.abs(want) + bound) + smallest(dtype)).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_both_gradients_in_one_call(score, normalize):
    x = make(300, 96, torch.float32, 5, masked=0.1, padded=0.1)
    w, ids = moe.route(x, 6, score, normalize)
    b = moe.balance(x, ids, score)
    dw = torch.randn((300, 6), generator=torch.Generator().manual_seed(1)).cuda()
    d_loss = torch.full((1,), 3.0, device="cuda")
    d = moe.route_grad(dw, x, ids, score, normalize, balance=(d_loss, b))
    v, i, slope = doubles(x), ids.cpu().numpy(), doubles(b.slope)
    want = oracle.route_grad(doubles(dw), v, i, score, normalize) + oracle.balance_grad(3.0, v, slope, score)
    p = oracle.probabilities(v, score)
    bound = grad_bound(v, doubles(dw), i, score, normalize)
    bound = bound + 3.0 * p * (slope + (p * slope).sum(1, keepdims=True)) * (2 * spread(v) + 180) * E
    if (score, normalize) == ("softmax", False):  # one sum of both over the row, taken off every expert
        bound = bound + p * (3.0 * (p * slope).sum(1, keepdims=True)) * (2 * spread(v) + 180) * E
    assert (np.abs(doubles(d) - want) <= bound + 2 * E * (np.abs(want) + bound) + 2.0 ** -140).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_gradients_against_differences(score, normalize):
    """Central differences of the forward calls.  With step h the formula's third derivative adds at most h^2 / 6 times
    6 sum |g| (a score's derivatives are below 1, 1, 6), and the values' errors (D + 60) E sum |g| / h."""
    x = make(4, 12, torch.float32, 9)
    ids = moe.route(x, 3, score, normalize)[1]
    g = torch.randn((4, 3), generator=torch.Generator().manual_seed(2)).cuda()
    d = doubles(moe.route_grad(g, x, ids, score, normalize))
    b = moe.balance(x, ids, score)
    db = doubles(moe.balance_grad(torch.ones((), device="cuda"), x, b, score))
    h = 2.0 ** -6
    big, slope = doubles(g), doubles(b.slope)
    for t in range(4):
        for e in range(12):
            ends, losses = [], []
            for sign in (1, -1):
                y = x.clone()
                y[t, e] += sign * h
                w = doubles(moe.route(y, 12, score, True)[0]) * 0  # (a full routing of the moved row runs as well)
                w, now = moe.route(y, 12, score, False)
                w, now = doubles(w)[t], now.cpu().numpy()[t]
                s = np.zeros(12)
                s[now] = w
                mine = s[ids.cpu().numpy()[t]]
                ends.append((big[t] * (mine / mine.sum() if normalize else mine)).sum())
                losses.append(float(moe.balance(y, ids, score).loss))
            step = float(x[t, e] + h) - float(x[t, e] - h)
            bound = (h * h + 200 * E / h) * 4 * np.abs(big[t]).sum()
            assert abs((ends[0] - ends[1]) / step - d[t, e]) <= bound
            bound = (h * h * slope.sum() + 400 * E * abs(float(b.loss)) / h) * 2
            assert abs((losses[0] - losses[1]) / step - db[t, e]) <= bound


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_logits_go_by_expert(dtype):
    x = torch.zeros((3, 300), dtype=dtype, device="cuda")
    x[1, 7] = -0.0
    x[2, ::3] = 1.0
    w, ids = check_route(x, 5, "softmax", True)
    assert ids.tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 3, 6, 9, 12]]
    assert (w == 0.2).all()


@pytest.mark.parametrize("experts,k", [(8, 3), (32, 4), (64, 8), (100, 16), (128, 20), (256, 8), (300, 8), (1024, 64)])
def test_logits_that_differ_in_their_last_bits(experts, k):
    """fp32 logits within a few of their last steps of each other, equal ones among them, next to far ones: the order is
    that of the values, then of the experts."""
    rng = np.random.default_rng(experts)
    rows = []
    for base in (1.0, -1.0, 3.0e-39, 1.7e38, -2.5):
        bits = np.full(experts, np.float32(base).view(np.int32)) + rng.integers(0, 9, experts).astype(np.int32)
        rows.append(bits.view(np.float32))
        far = rows[-1].copy()
        far[rng.random(experts) < 0.7] = np.float32(base) - np.float32(abs(base))  # (few near the top)
        rows.append(far)
    x = torch.from_numpy(np.stack(rows)).cuda()
    _, ids = moe.route(x, k)
    assert np.array_equal(ids.cpu().numpy(), oracle.choose(doubles(x), k))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score,normalize", KINDS)
def test_rows_with_little_or_nothing_left(dtype, score, normalize):
    x = torch.full((5, 70), -np.inf, dtype=dtype)
    x[1, 69] = -2.0
    x[2, 3], x[2, 40] = 1.0, torch.finfo(dtype).min
    x[3] = torch.finfo(dtype).min  # as a mask of the type's lowest value leaves it: all alike
    x[4, 10:12] = torch.finfo(dtype).max
    x = x.cuda()
    w, ids = moe.route(x, 3, score, normalize)
    i = ids.cpu().numpy()
    assert i.tolist() == [[-1] * 3, [69, -1, -1], [3, 40, -1], [0, 1, 2], [10, 11, -1]]
    want = oracle.weights(doubles(x), i, score, normalize)
    if score == "sigmoid" and normalize:
        want[3] = 1 / 3  # (sigmoids far below the smallest double)
    assert (np.abs(doubles(w) - want) <= 64 * E * want + 2.0 ** -126).all()
    d = moe.route_grad(torch.ones_like(w), x, ids, score, normalize)
    assert torch.isfinite(d).all() and (d[x == -np.inf] == 0).all()
    b = moe.balance(x, ids, score)
    assert torch.isfinite(b.loss) and int(b.counts.sum()) == 8
    d = moe.balance_grad(torch.ones((), device="cuda"), x, b, score)
    assert torch.isfinite(d).all() and (d[x == -np.inf] == 0).all()


def test_scores_of_very_low_logits_keep_their_proportions():
    x = torch.tensor([[-200.0, -201.0, -300.0, -203.0]], device="cuda")
    w, ids = moe.route(x, 3, "sigmoid")
    want = np.exp([0.0, -1.0, -3.0])
    assert ids.tolist() == [[0, 1, 3]] and np.allclose(doubles(w)[0], want / want.sum(), rtol=70 * E, atol=0)
    b = moe.balance(x, ids, "sigmoid")  # p = softmax here: 4 / 3 (1 - p[2])
    assert abs(float(b.loss) - 4 / 3) <= 300 * E


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_infinity_show(dtype):
    x = make(6, 50, dtype, 3)
    x[1, 20] = np.nan
    x[2, 5], x[2, 30] = np.inf, np.nan
    x[3, 8] = np.inf
    x[4, 49] = -np.nan
    x[5] = -np.inf
    x[5, 13] = np.nan
    w, ids = moe.route(x, 4)
    assert ids[1, 0] == 20 and ids[2, :2].tolist() == [30, 5] and ids[3, 0] == 8 and ids[4, 0] == 49 and ids[5].tolist() == [13, -1, -1, -1]
    assert torch.isfinite(w[0]).all() and torch.isnan(w[1:5]).all() and torch.isnan(w[5, 0]) and (w[5, 1:] == 0).all()
    w, _ = moe.route(x, 4, "sigmoid", False)
    assert torch.isnan(w[1, 0]) and torch.isfinite(w[1, 1:]).all() and w[3, 0] == 1
    assert torch.isnan(moe.balance(x, ids).loss) and torch.isfinite(moe.balance(x[:1], ids[:1]).loss)
    dw = torch.ones_like(w)
    d = moe.route_grad(dw, x, ids)
    assert torch.isfinite(d[0]).all() and torch.isnan(d[1, 20]) and torch.isnan(d[5, 13])


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("k", [5, 40])
def test_the_same_expert_twice_adds_both(score, normalize, k):
    x = make(20, 64, torch.float32, 4)
    rng = np.random.default_rng(k)
    ids = rng.integers(-1, 4, (20, k)).astype(np.int32)
    dw = torch.randn((20, k), generator=torch.Generator().manual_seed(6)).cuda()
    t = torch.from_numpy(ids).cuda()
    d = moe.route_grad(dw, x, t, score, normalize)
    v = doubles(x)
    want = oracle.route_grad(doubles(dw), v, ids, score, normalize)
    bound = grad_bound(v, doubles(dw), ids, score, normalize)
    assert (np.abs(doubles(d) - want) <= bound + (1 + k) * E * bound.max()).all()
    assert torch.equal(d, moe.route_grad(dw, x, t, score, normalize))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts,pitch,at", [(64, 65, 0), (64, 72, 1), (40, 48, 8), (256, 264, 4), (129, 200, 3)])
def test_strides_and_starts(dtype, experts, pitch, at):
    x = make(50, experts, dtype, 8, pitch=pitch, at=at)
    c = x.contiguous()
    w, ids = moe.route(x, 6)
    w2, ids2 = moe.route(c, 6)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    dw = torch.rand((50, 12), device="cuda")[:, ::2]
    b, b2 = moe.balance(x, ids), moe.balance(c, ids)
    assert all(torch.equal(p, q) for p, q in zip(b, b2))
    one = torch.ones((), device="cuda")
    assert torch.equal(moe.route_grad(dw, x, ids, balance=(one, b)), moe.route_grad(dw.contiguous(), c, ids, balance=(one, b)))
    cols = c.t().contiguous().t()  # columns one after the other
    assert torch.equal(moe.route(cols, 6)[1], ids)


def test_counts_are_those_of_a_plan():
    x = make(4000, 96, torch.bfloat16, 11, padded=0.1)
    _, ids = moe.route(x, 8)
    plan = moe.sort(ids, 96)
    assert torch.equal(moe.balance(x, ids).counts, plan.offsets[1:] - plan.offsets[:-1])


def test_equal_inputs_give_equal_bits():
    x = make(9000, 128, torch.bfloat16, 12)
    w, ids = moe.route(x, 8)
    one = torch.ones((), device="cuda")
    first = moe.balance(x, ids)
    for _ in range(5):
        b = moe.balance(x, ids)
        assert all(torch.equal(p, q) for p, q in zip(first, b))
        assert torch.equal(moe.route_grad(w, x, ids, balance=(one, b)), moe.route_grad(w, x, ids, balance=(one, first)))


def test_loss_of_an_even_routing_is_one():
    x = torch.zeros((64, 16), device="cuda")
    ids = torch.arange(64 * 4, dtype=torch.int32, device="cuda").view(64, 4) % 16
    b = moe.balance(x, ids)
    assert abs(float(b.loss) - 1) <= 300 * E and (b.counts == 16).all()


def test_streams_and_graphs():
    """On a stream of its own, and captured with replays on new contents."""
    x = make(600, 64, torch.bfloat16, 13)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    one = torch.ones((), device="cuda")

    def step(stream=None):
        w, ids = moe.route(x, 4, stream=stream)
        b = moe.balance(x, ids, stream=stream)
        return w, ids, *b, moe.route_grad(w, x, ids, balance=(one, b), stream=stream)

    want = step()
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in (20, 21):
        x.copy_(make(600, 64, torch.bfloat16, seed, padded=0.3))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, step()))


def test_rows_past_32_bit_offsets():
    """The last rows of 4.2 million x 1024 logits (8.6 GB), and of their gradient."""
    tokens, experts = (1 << 22) + 7, 1024
    x = torch.zeros((tokens, experts), dtype=torch.bfloat16, device="cuda")
    tail = make(5, experts, torch.bfloat16, 3)
    x[-5:] = tail
    w, ids = moe.route(x, 2)
    w2, ids2 = moe.route(tail, 2)
    assert torch.equal(w[-5:], w2) and torch.equal(ids[-5:], ids2) and (ids[:-5] == torch.tensor([0, 1], device="cuda")).all()
    b = moe.balance(x, ids)
    assert int(b.counts.sum()) == 2 * tokens
    d = moe.route_grad(torch.ones_like(w), x, ids, balance=(torch.ones((), device="cuda"), b))
    assert torch.equal(d[-5:], moe.route_grad(torch.ones_like(w2), tail, ids2, balance=(torch.ones((), device="cuda"), b)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts", [32, 64, 100, 128, 256])
def test_all_chosen_logits_in_one_lane(experts, dtype):
    """A lane holds eight neighbouring columns of 16 bits, or four and the four half a row of lanes further on."""
    half = max(16, 1 << (experts - 1).bit_length() - 1)
    x = make(64, experts, dtype, 5)
    for t in range(64):
        first = t * 4 % (experts - 8)
        cols = [c for c in range(first // 8 * 8, first // 8 * 8 + 8)] if t % 2 else \
            [c for c in range(first % half, first % half + 4)] + [c + half for c in range(first % half, first % half + 4) if c + half < experts]
        x[t, cols] = torch.linspace(20, 30 + t % 3, len(cols), device="cuda").to(dtype)
    for k in (1, 7, 8, 9, 16):
        check_route(x, k, "softmax", True)


@pytest.mark.parametrize("experts,k", [(64, 8), (256, 8), (256, 5), (40, 6), (1000, 8), (256, 40), (64, 64)])
def test_fp32_logits_that_are_close(experts, k):
    """Values a step or a few apart, in groups that the choice cuts through, and equal ones."""
    rng = np.random.default_rng(experts + k)
    x = np.repeat(rng.standard_normal((200, -(-experts // 5))).astype(np.float32), 5, 1)[:, :experts]
    steps = rng.integers(-3, 4, x.shape) * (rng.random((200, 1)) < 0.7)
    x = (x.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    x = rng.permuted(x, axis=1)
    check_route(torch.from_numpy(x).cuda(), k, "softmax", True)
    check_route(torch.from_numpy(x).cuda(), k, "sigmoid", False)


# The largest batches of one CTA, one more, the largest of a cluster, one more: by the experts of a row.
@pytest.mark.parametrize("tokens,experts,k", [(512, 20, 3), (513, 20, 3), (4096, 32, 1), (4097, 32, 9), (257, 64, 8), (2048, 40, 6),
                                              (2049, 64, 2), (129, 100, 5), (1024, 128, 3), (1025, 128, 3), (65, 256, 8),
                                              (512, 200, 40), (513, 256, 8), (33, 1000, 8), (256, 1024, 64), (257, 999, 2)])
@pytest.mark.parametrize("score,dtype", [("softmax", torch.bfloat16), ("sigmoid", torch.float32)])
def test_balance_by_one_cta_a_cluster_or_two_kernels(tokens, experts, k, score, dtype):
    x = make(tokens, experts, dtype, tokens + k, masked=0.1, padded=0.2)
    ids = np.random.default_rng(tokens).integers(-1, experts + 1, (tokens, k)).astype(np.int32)
    b = moe.balance(x, torch.from_numpy(ids).cuda(), score)
    v = doubles(x)
    loss, counts, slope = oracle.balance(v, ids, score)
    assert np.array_equal(b.counts.cpu().numpy(), counts) and (np.abs(doubles(b.slope) - slope) <= E * slope).all()
    assert abs(float(b.loss) - loss) <= (spread(v).max() + 260 + tokens / 16) * E * loss
    again = moe.balance(x, torch.from_numpy(ids).cuda(), score)
    assert all(torch.equal(p, q) for p, q in zip(b, again))


def test_balance_of_more_rows_than_fp32_counts():
    """2^24 + 3 rows, whose number is no fp32 value; all but one use expert 1, so p is 1/3, 2/3 and 0, 1 in the last."""
    tokens = (1 << 24) + 3
    x = torch.tensor([0.0, np.log(2.0)], dtype=torch.float32, device="cuda").repeat(tokens, 1)
    x[-1, 0] = -np.inf
    ids = torch.ones((tokens, 1), dtype=torch.int32, device="cuda")
    ids[5] = 0
    b = moe.balance(x, ids)
    assert b.counts.tolist() == [1, tokens - 1]
    slope = 2.0 * np.array([1, tokens - 1]) / (float(tokens) * tokens)
    assert (np.abs(doubles(b.slope) - slope) <= E * slope).all()
    p = np.exp(doubles(x[:1])[0])
    p /= p.sum()
    loss = slope[0] * p[0] * (tokens - 1) + slope[1] * (p[1] * (tokens - 1) + 1)
    # A spread of 1; a lane of 152 CTAs' 256 rows at a time adds 432 values, and 200 additions join the lanes.
    assert abs(float(b.loss) - loss) <= (1 + 60 + 432 + 200) * E * loss


# From 20 tokens for each of 152 SMs on, with up to 16 slots on rows of more than 128 logits (or more slots than a row's
# lanes), a warp takes the slots of several tokens at once: sizes around that, every number of slots that share a warp,
# slots without an expert, of an expert that the token may not use, and of the same expert twice.
@pytest.mark.parametrize("score,normalize,dtype", [("softmax", True, torch.bfloat16), ("softmax", True, torch.float32),
                                                   ("sigmoid", True, torch.float16), ("sigmoid", False, torch.float32)])
@pytest.mark.parametrize("tokens,experts,k", [(3039, 130, 8), (3041, 130, 1), (3050, 200, 3), (3047, 256, 4), (3333, 256, 8),
                                              (3041, 199, 9), (4001, 257, 16), (3042, 1000, 5), (3100, 40, 16), (3101, 64, 9)])
@pytest.mark.parametrize("odd_slots", [False, True])
def test_gradients_of_many_tokens(tokens, experts, k, score, normalize, dtype, odd_slots):
    x = make(tokens, experts, dtype, tokens + k, masked=0.2, padded=0.05, pitch=experts + 3, at=1) if k % 2 else \
        make(tokens, experts, dtype, tokens + k, masked=0.2, padded=0.05)
    w, ids = moe.route(x, k, score, normalize)
    b = moe.balance(x, ids, score)
    if odd_slots:
        ids = torch.randint(-2, experts + 2, (tokens, k), generator=torch.Generator().manual_seed(tokens)).int().cuda()
        ids[::3, -1] = ids[::3, 0]
    dw = torch.randn((tokens, k), generator=torch.Generator().manual_seed(k)).cuda()
    v, i, slope = doubles(x), ids.cpu().numpy(), doubles(b.slope)
    i = np.where((i >= 0) & (i < experts) & (np.take_along_axis(v, i.clip(0, experts - 1), 1) > -np.inf), i, -1)
    want = oracle.route_grad(doubles(dw), v, i, score, normalize)
    bound = grad_bound(v, doubles(dw), i, score, normalize)
    if odd_slots:  # one addition for each further slot of an expert, at most k
        bound = bound * (1 + k * E)
    d = moe.route_grad(dw, x, ids, score, normalize)
    assert (np.abs(doubles(d) - want) <= bound + half_ulp(dtype) * (np.abs(want) + bound) + smallest(dtype)).all()
    d = moe.route_grad(dw, x, ids, score, normalize, balance=(torch.full((), 3.0, device="cuda"), b))
    p = oracle.probabilities(v, score)
    want = want + oracle.balance_grad(3.0, v, slope, score)
    bound = bound + 3.0 * p * (slope + (p * slope).sum(1, keepdims=True)) * (2 * spread(v) + 180) * E
    bound = bound + 2 * E * (np.abs(want) + bound)
    assert (np.abs(doubles(d) - want) <= bound + half_ulp(dtype) * (np.abs(want) + bound) + smallest(dtype)).all()


def test_kernel_times_go_by_their_ids():
    x = make(3000, 64, torch.bfloat16, 1)
    one = torch.ones((), device="cuda")
    zc.zc_timing_enable(1)
    try:
        zc.zc_timing_collect()
        w, ids = moe.route(x, 4)
        b = moe.balance(x, ids)
        moe.route_grad(w, x, ids, balance=(one, b))
        torch.cuda.synchronize()
        seen = [k for k, ms in zc.zc_timing_collect() if ms > 0]
    finally:
        zc.zc_timing_enable(0)
    assert seen == [zc.ZC_KERNEL_MOE_ROUTE, zc.ZC_KERNEL_MOE_BALANCE, zc.ZC_KERNEL_MOE_BALANCE, zc.ZC_KERNEL_MOE_ROUTE_GRAD]


def test_two_streams_at_once():
    """Calls of the same sizes on two streams, each with a workspace of its own."""
    xs = [make(5000, 64, torch.bfloat16, s) for s in (1, 2)]
    ids = [moe.route(x, 4)[1] for x in xs]
    want = [moe.balance(x, i) for x, i in zip(xs, ids)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for x, i, s in zip(xs, ids, streams):
            got.append(moe.balance(x, i, stream=s))
    torch.cuda.synchronize()
    for n, b in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(b, want[n % 2]))


def test_refusals():
    x = torch.zeros((4, 8), device="cuda")
    w, ids = moe.route(x, 2)
    b = moe.balance(x, ids)
    one = torch.ones((), device="cuda")
    with pytest.raises(ValueError):
        moe.route(x, 9)
    with pytest.raises(ValueError):
        moe.route(x, 0)
    with pytest.raises(ValueError):
        moe.route(x, 2, "tanh")
    with pytest.raises(ValueError):
        moe.route(x[0], 2)
    with pytest.raises(TypeError):
        moe.route(x.double(), 2)
    with pytest.raises(ValueError):
        moe.route(torch.zeros((2, 1025), device="cuda"), 2)
    with pytest.raises(TypeError):
        moe.balance(x, ids.long())
    with pytest.raises(ValueError):
        moe.balance(x[:3], ids)
    with pytest.raises(ValueError):
        moe.route_grad(w[:, :1], x, ids)
    with pytest.raises(TypeError):
        moe.route_grad(w.half(), x, ids)
    with pytest.raises(TypeError):
        moe.route_grad(None, x, ids)
    with pytest.raises(ValueError):
        moe.balance_grad(torch.ones(2, device="cuda"), x, b)
    with pytest.raises(ValueError):
        moe.balance_grad(one, x[:, :5], b)
    with pytest.raises(TypeError):
        moe.balance_grad(None, x, b)
    with pytest.raises(TypeError):
        moe.route(x.cpu(), 2)
    with pytest.raises(RuntimeError, match="requires a gradient"):
        moe.route(x.clone().requires_grad_(), 2)
    with torch.no_grad():
        moe.route(x.clone().requires_grad_(), 2)


def test_no_tokens():
    x = torch.zeros((0, 16), dtype=torch.bfloat16, device="cuda")
    w, ids = moe.route(x, 4)
    b = moe.balance(x, ids)
    assert w.shape == ids.shape == (0, 4) and float(b.loss) == 0 and int(b.counts.sum()) == 0 and float(b.slope.abs().sum()) == 0
    assert moe.route_grad(w, x, ids, balance=(torch.ones((), device="cuda"), b)).shape == (0, 16)
