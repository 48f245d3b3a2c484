"""The entry points of include/zc_router.h and include/zc_int4.h without a GPU: exported, bound with the headers' arguments,
and refusing what the headers say they refuse.  And the oracle's gradients, against differences of its own forward."""
import os
import re

import numpy as np
import pytest

import router_oracle as oracle
from lossless_bf16_compression_gb300 import binding as zc
from lossless_bf16_compression_gb300 import build as zbuild

torch = pytest.importorskip("torch")
from lossless_bf16_compression_gb300 import _tensors  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30  # aligned fake addresses, far apart; never dereferenced by calls that are refused
B, C, D, E, F = (A * i for i in range(2, 7))
INV, MIS = zc.ZC_ERR_INVALID_ARG, zc.ZC_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def _built():
    zbuild.build()


def header(name):
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)


@pytest.mark.parametrize("name,table", [("zc_router.h", "ROUTER_SIGNATURES"), ("zc_int4.h", "INT4_SIGNATURES")])
def test_every_declared_symbol_is_bound_with_its_arguments(name, table):
    table = getattr(_tensors, table)
    found = re.findall(r"^\s*(?:size_t|int)\s+(zc_\w+)\s*\(([^)]*)\)", header(name), flags=re.M)
    assert sorted(n for n, _ in found) == sorted(table)
    for symbol, args in found:
        kinds = ["p" if "*" in a or "cudaStream_t" in a else "n" if "size_t" in a else "f" if "float" in a else "i" for a in args.split(",")]
        bound = [{_tensors._P: "p", _tensors._N: "n", _tensors._I: "i", _tensors._F: "f"}[t] for t in table[symbol][1]]
        assert kinds == bound, symbol
        assert hasattr(zc.lib(), symbol)


def test_constants_match_the_headers():
    from lossless_bf16_compression_gb300 import int4, moe

    d = {}
    for name in ("zc.h", "zc_moe.h", "zc_router.h", "zc_int4.h"):
        d |= dict(re.findall(r"^#define\s+(ZC_\w+)\s+(\d+)\s*$", header(name), flags=re.M))
    assert moe.SCORES == {"softmax": int(d["ZC_SCORE_SOFTMAX"]), "sigmoid": int(d["ZC_SCORE_SIGMOID"])}
    assert int4.GROUP == int(d["ZC_INT4_GROUP"]) and int4.ROWS == int(d["ZC_INT4_ROWS"])
    ids = {k: int(v) for k, v in d.items() if k.startswith("ZC_KERNEL_")}
    assert len(set(ids.values())) == len(ids) == 24
    for name, value in ids.items():
        assert getattr(zc, name) == value, name


def refused(name, args, changes):
    fn = _tensors.fn(name)
    for at, value, code in changes:
        bad = list(args)
        bad[at] = value
        assert fn(*bad) == code, (name, at, value)
    if not os.path.exists("/dev/nvidia0"):
        assert fn(*args) == zc.ZC_ERR_CUDA  # valid arguments reach the runtime, which has no device


def test_route_refuses():
    refused("zc_moe_route", [A, 64, 0, 10, 64, 8, 0, 1, 1.0, B, C, 0],
            [(0, 0, INV), (1, 63, INV), (2, 3, INV), (4, 0, INV), (4, 1025, INV), (5, 0, INV), (5, 65, INV), (6, 2, INV),
             (6, -1, INV), (9, 0, INV), (10, 0, INV), (0, A + 1, MIS), (9, B + 2, MIS), (10, C + 1, MIS), (9, A + 64, INV),
             (10, B + 8, INV), (3, 1 << 30, INV)])
    refused("zc_moe_route", [A, 5, 0, 10, 5, 5, 0, 1, 1.0, B, C, 0], [(5, 6, INV)])  # more than there are


def test_balance_refuses():
    assert _tensors.fn("zc_moe_balance_workspace")(0, 8) == 0 == _tensors.fn("zc_moe_balance_workspace")(10, 0)
    assert _tensors.fn("zc_moe_balance_workspace")(100000, 64) > 0 == _tensors.fn("zc_moe_balance_workspace")(100000, 1025)
    refused("zc_moe_balance", [A, 64, 0, B, 100000, 64, 8, 0, C, D, E, F, 0],
            [(0, 0, INV), (1, 63, INV), (2, -1, INV), (3, 0, INV), (5, 0, INV), (6, 0, INV), (6, 65, INV), (7, 2, INV),
             (8, 0, INV), (9, 0, INV), (10, 0, INV), (11, 0, INV), (0, A + 1, MIS), (3, B + 2, MIS), (8, C + 2, MIS),
             (9, D + 2, MIS), (10, E + 2, MIS), (11, F + 8, MIS), (8, A, INV), (9, B, INV), (10, D + 4, INV), (11, A + 16, INV)])


def test_route_grad_refuses():
    args = [A, B, C, D, E, 64, 0, 10, 64, 8, 0, 1, 1.0, F, 64, 0]
    refused("zc_moe_route_grad", args,
            [(0, 0, INV), (1, 0, INV), (2, 0, INV), (3, 0, INV), (4, 0, INV), (5, 63, INV), (6, 3, INV), (8, 0, INV), (9, 0, INV),
             (10, 2, INV), (13, 0, INV), (14, 63, INV), (0, A + 1, MIS), (1, B + 2, MIS), (2, C + 2, MIS), (3, D + 2, MIS),
             (4, E + 1, MIS), (13, F + 1, MIS), (13, E, INV), (13, A, INV), (13, D, INV)])
    neither = list(args)
    neither[0] = neither[1] = neither[2] = neither[3] = 0
    assert _tensors.fn("zc_moe_route_grad")(*neither) == INV


def test_int4_refuses():
    refused("zc_int4_quantize", [A, 0, 2, 64, 256, B, C, 0],
            [(0, 0, INV), (1, 3, INV), (2, 0, INV), (2, 1025, INV), (3, 0, INV), (4, 0, INV), (4, (1 << 20) + 1, INV), (5, 0, INV),
             (6, 0, INV), (0, A + 1, MIS), (5, B + 8, MIS), (6, C + 8, MIS), (5, A, INV), (6, B + 16, INV)])
    refused("zc_int4_values", [A, B, 2, 64, 256, 0, C, 0],
            [(0, 0, INV), (1, 0, INV), (2, 0, INV), (3, 0, INV), (4, 0, INV), (5, 3, INV), (6, 0, INV), (0, A + 8, MIS), (1, B + 8, MIS),
             (6, C + 1, MIS), (6, A + 16, INV), (6, B, INV)])
    refused("zc_int4_matmul", [A, 256, 0, 10, B, C, 2, 64, 256, D, E, 64, 0, 0],
            [(0, 0, INV), (1, 255, INV), (2, 3, INV), (3, 1 << 31, INV), (4, 0, INV), (5, 0, INV), (6, 0, INV), (7, 0, INV), (8, 0, INV),
             (9, 0, INV), (10, 0, INV), (11, 63, INV), (12, 3, INV), (0, A + 1, MIS), (4, B + 8, MIS), (5, C + 8, MIS),
             (9, D + 2, MIS), (10, E + 1, MIS), (10, A, INV), (10, B, INV), (10, C, INV), (10, D, INV)])


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="checks the no-GPU failure path")
def test_tensors_on_the_cpu_are_refused():
    from lossless_bf16_compression_gb300 import int4, moe

    x, ids = torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int32)
    b = moe.Balance(x[0, 0], ids[0], x[0])
    for call in (lambda: moe.route(x, 2), lambda: moe.balance(x, ids), lambda: moe.route_grad(x[:, :2], x, ids),
                 lambda: moe.balance_grad(x[0, :1], x, b), lambda: int4.quantize_weight(x),
                 lambda: int4.Matrix(torch.zeros((1, 1, 1024), dtype=torch.uint8), torch.ones((1, 1, 16)).bfloat16(), 2, 8).values(),
                 lambda: int4.matmul(x, None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        moe.route(x, 2, "tanh")


def test_the_layout_of_records_is_one_to_one():
    rng = np.random.default_rng(1)
    q, s = rng.integers(-7, 8, (37, 2, 128)), rng.integers(128, 256, (37, 2)).astype(float)
    data, scales = oracle.pack(q, s)
    q2, s2, rest, one = oracle.unpack(data, scales, 37, 256)
    assert np.array_equal(q, q2) and np.array_equal(s, s2) and (rest == 0).all() and (one == 1).all()


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_the_oracle_s_gradients_are_differences_of_its_forward(score, normalize):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 7)) * 2
    ids = oracle.choose(x, 3)
    ids[1, 2] = -1
    g = rng.standard_normal((3, 3))
    d = oracle.route_grad(g, x, ids, score, normalize, 1.5)
    loss, counts, slope = oracle.balance(x, ids, score)
    db = oracle.balance_grad(1.0, x, slope, score)
    h = 1e-5
    for t in range(3):
        for e in range(7):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            slow = [(g * oracle.weights(y, ids, score, normalize, 1.5)).sum() for y in (up, down)]
            assert abs((slow[0] - slow[1]) / (2 * h) - d[t, e]) < 1e-8
            slow = [oracle.balance(y, ids, score)[0] for y in (up, down)]
            assert abs((slow[0] - slow[1]) / (2 * h) - db[t, e]) < 1e-8
