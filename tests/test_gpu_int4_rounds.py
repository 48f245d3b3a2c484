"""Products on 4-bit weights whose CTAs have several rounds: of one pass and of the next, with x whole in shared memory and
in parts, with warps that share a round's lines; and offsets that do not fit, with what lies around the rows.

``rounds`` restates how the list of lines is cut (16 warps, two record rows to a line, 226 KB of shared memory), so that the
sizes can be seen to reach what they are for, without a GPU.  Results are compared with 64-bit products of the weights'
own values (which are exact in fp32 and tested by themselves), to the bound of the products' other tests, and with a second call.
"""
import pytest

from gpu_helpers import require_gpu
from moe_oracle import half_ulp, smallest

torch = pytest.importorskip("torch")

from lossless_bf16_compression_gb300 import binding as zc  # noqa: E402
from lossless_bf16_compression_gb300 import int4  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]
WARPS, SMS = 16, 152


def rounds(counts, n, k, dtype, sms=SMS):
    """For each CTA its rounds: (pass, whether x lies there whole, first line, lines, columns of eight)."""
    parts, rows, groups = 3 if dtype == torch.float32 else 1, sum(counts), len(counts)
    nt = 1 if rows * parts <= 8 else 2
    each, blocks, lines = 8 * nt // parts, -(-k // 128), -(-(-(-n // 16)) // 2)
    room = (226 * 1024 - 20480 * nt - 8 * (groups + 1)) // 2048 // (2 * nt) * (2 * nt)
    room = min(room, blocks * nt)
    passes = [min(each, c - a) for c in counts for a in range(0, c, each)]
    columns = [-(-r * parts // 8) for r in passes]
    bound = [0]
    for c in columns:
        bound.append(bound[-1] + (2 + c) * lines)
    total = bound[-1]

    def line_at(point):  # of all passes
        if point >= total:
            return len(passes) * lines
        p = max(i for i in range(len(passes)) if bound[i] <= point)
        return p * lines + (point - bound[p]) // (2 + columns[p])

    most = (rows * parts + 8 * nt - 1) // (8 * nt) + min(groups, rows)
    ctas = min(most * -(-n // 16), sms)
    share, more = divmod(total, ctas)
    out = []
    for b in range(ctas):
        begin, end = (line_at(share * c + min(c, more)) for c in (b, b + 1))
        mine = []
        while begin < end:
            p, at = divmod(begin, lines)
            take = min(WARPS, end - begin, lines - at)
            if WARPS // 2 < take < WARPS * 3 // 4:
                take = WARPS // 2
            mine.append((p, blocks <= room // columns[p], at, take, columns[p]))
            begin += take
        out.append(mine)
    return out


def kinds(all_rounds):
    """What the rounds of all CTAs contain, by name."""
    seen = set()
    for mine in all_rounds:
        for i, (p, whole, at, lines, columns) in enumerate(mine):
            x = ("whole" if whole else "parts") + f" {columns}"
            if i and mine[i - 1][0] == p:
                before = WARPS // mine[i - 1][3] > 1
                seen.add(f"{x}, again after {'shared' if before else 'own'}, now {'shared' if WARPS // lines > 1 else 'own'}")
            elif i:
                seen.add(f"{'whole' if mine[i - 1][1] else 'parts'} {mine[i - 1][4]} to {x}")
    return seen


# counts of rows, n, k: what they are for
CASES = [
    # 19 to 22 lines a CTA, x whole
    ([40], 30000, 200, [torch.bfloat16, torch.float16],
     {"whole 2, again after own, now shared", "whole 1, again after own, now shared", "whole 2 to whole 2", "whole 2 to whole 1"}),
    ([2], 156000, 130, [torch.float32], {"whole 1, again after own, now own", "whole 1, again after own, now shared"}),
    # nine to eleven lines a CTA: eight, two warps to each, and the rest
    ([5, 7, 3, 9, 12], 10000, 640, [torch.bfloat16], {"whole 2, again after shared, now shared", "whole 1, again after shared, now shared"}),
    # more than 16 rows of x or more columns than its place holds: in parts
    ([10, 0, 16, 3, 9, 20, 11], 8000, 7300, [torch.bfloat16, torch.float16],
     {"parts 2, again after shared, now shared", "parts 2 to parts 2", "parts 2 to whole 1", "whole 1 to parts 2"}),
    ([33], 44000, 6100, [torch.bfloat16], {"parts 2, again after own, now shared", "parts 2 to whole 1"}),
    ([5, 3, 9, 4], 8000, 7301, [torch.float32], {"parts 2, again after shared, now shared", "parts 2 to parts 2"}),
    # eight columns at a time at most
    ([6], 48100, 14000, [torch.bfloat16, torch.float16], {"parts 1, again after shared, now shared"}),
    ([3, 2, 1], 30000, 13500, [torch.bfloat16], {"parts 1, again after own, now shared", "parts 1 to parts 1"}),
    ([2], 48100, 13101, [torch.float32], {"parts 1, again after shared, now shared"}),
]
RUNS = [(counts, n, k, dtype, want) for counts, n, k, dtypes, want in CASES for dtype in dtypes]


@pytest.mark.parametrize("counts,n,k,dtype,want", RUNS)
def test_the_sizes_reach_their_rounds(counts, n, k, dtype, want):
    seen = kinds(rounds(counts, n, k, dtype))
    assert want <= seen, (want - seen, seen)


def weights(groups, n, k, seed):
    """Random weights of -7 .. 7 with random scales, records and all; columns past k and rows past n hold some too, which
    no result may show."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (groups, -(-n // 16), -(-k // 128))
    low, high = (torch.randint(1, 16, (*shape, 1024), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    scales = (torch.rand((*shape, 16), generator=g, device="cuda") + 1) / 64
    return int4.Matrix(low | high << 4, scales.bfloat16(), n, k)


def check(x, m, counts, y):
    at, values, slices = 0, m.values(), -(-m.cols // 128)
    for g, c in enumerate(counts):
        for first in range(0, m.rows, 4096) if c else ():
            w = values[g, first:first + 4096].double()
            rows = x[at:at + c].double()
            want, size = rows @ w.t(), rows.abs() @ w.abs().t()
            bound = size * (3 * 128 * 2.0 ** -23 + (2 * slices + 40) * 2.0 ** -24)
            bound = bound + half_ulp(y.dtype) * (want.abs() + bound) + smallest(y.dtype)
            assert ((y[at:at + c, first:first + 4096].double() - want).abs() <= bound).all(), (g, first)
        at += c
    assert (y[at:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,n,k,dtype,want", RUNS)
def test_several_rounds(counts, n, k, dtype, want):
    require_gpu()
    zc.status(reset=True)
    m = weights(len(counts), n, k, n + k)
    g = torch.Generator(device="cuda").manual_seed(k)
    offsets = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn((sum(counts), k), generator=g, device="cuda").to(dtype)
    y = int4.matmul(x, m, offsets)
    check(x, m, counts, y)
    for _ in range(3):
        assert torch.equal(int4.matmul(x, m, offsets), y)
    assert zc.status(reset=True) == zc.ZC_OK


def bad_offsets(groups, rows, at, value):
    o = [rows * i // groups for i in range(groups + 1)]
    o[at] = value
    return o


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("groups,rows,at,value", [
    (3, 6, 0, 1), (3, 6, 1, 5), (3, 6, 3, 7), (3, 6, 1, -3), (3, 6, 2, 1 << 30), (40, 6, 40, 7), (40, 80, 35, -1), (40, 80, 33, 200),
    (40, 80, 0, 2), (600, 50, 600, 51), (600, 50, 590, -2 ** 31), (600, 50, 3, 2 ** 31 - 1), (1024, 9, 1000, 100)])
def test_offsets_that_do_not_fit_touch_nothing_else(groups, rows, at, value, dtype):
    """No row outside the output and nothing between its rows is written, and the status says so: wherever the wrong
    offset is, no group's rows are multiplied."""
    require_gpu()
    from lossless_bf16_compression_gb300 import _tensors

    n, k, pitch, guard = 40, 256, 48, 8
    m = weights(groups, n, k, groups)
    x = torch.full((rows + 2 * guard, k), float("nan"), dtype=dtype, device="cuda")
    x[guard:guard + rows] = 1.0
    out = torch.full((rows + 2 * guard, pitch), 5.0, dtype=dtype, device="cuda")
    offsets = torch.tensor(bad_offsets(groups, rows, at, value), dtype=torch.int32, device="cuda")
    zc.status(reset=True)
    kind = TYPES.index(dtype)
    rc = _tensors.fn("zc_int4_matmul")(x[guard:].data_ptr(), k, kind, rows, m.data.data_ptr(), m.scales.data_ptr(), groups, n, k,
                                       offsets.data_ptr(), out[guard:].data_ptr(), pitch, kind, torch.cuda.current_stream().cuda_stream)
    assert rc == zc.ZC_OK and zc.status(reset=True) == zc.ZC_ERR_CORRUPT
    assert (out[:guard] == 5).all() and (out[guard + rows:] == 5).all() and (out[:, n:] == 5).all()
    assert not torch.isnan(out).any()  # (rows beside x were not read into any)
    # The next call is not touched by it.
    good = torch.tensor(bad_offsets(groups, rows, 0, 0), dtype=torch.int32, device="cuda")
    y = int4.matmul(x[guard:guard + rows], m, good)
    counts = (good[1:] - good[:-1]).tolist()
    check(x[guard:guard + rows], m, counts, y)
    assert zc.status(reset=True) == zc.ZC_OK
