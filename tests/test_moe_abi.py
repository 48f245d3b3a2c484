"""The entry points of include/zc_moe.h without a GPU: exported, bound with the header's arguments, and refusing what
the header says they refuse."""
import os
import re

import pytest

from lossless_bf16_compression_gb300 import binding as zc
from lossless_bf16_compression_gb300 import build as zbuild

pytest.importorskip("torch")
from lossless_bf16_compression_gb300 import _tensors  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30  # aligned fake addresses, far apart; never dereferenced by calls that are refused
B, C, D, E, F = (A * i for i in range(2, 7))


@pytest.fixture(scope="module", autouse=True)
def _built():
    zbuild.build()


def header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "zc_moe.h")).read(), flags=re.S)


def test_every_declared_symbol_is_bound_with_its_arguments():
    found = re.findall(r"^\s*(?:size_t|int)\s+(zc_\w+)\s*\(([^)]*)\)", header(), flags=re.M)
    assert sorted(n for n, _ in found) == sorted(_tensors.SIGNATURES)
    for name, args in found:
        kinds = ["p" if "*" in a or "cudaStream_t" in a else "n" if "size_t" in a else "i" for a in args.split(",")]
        bound = [{_tensors._P: "p", _tensors._N: "n", _tensors._I: "i"}[t] for t in _tensors.SIGNATURES[name][1]]
        assert kinds == bound, name
        assert hasattr(zc.lib(), name)


def test_constants_match_the_header():
    d = dict(re.findall(r"^#define\s+(ZC_\w+)\s+(\d+)\s*$", header(), flags=re.M))
    assert int(d["ZC_MOE_MAX_EXPERTS"]) == _tensors.MAX_EXPERTS and int(d["ZC_MOE_MAX_K"]) == _tensors.MAX_K
    assert sorted(_tensors.TYPES.values()) == [int(d[f"ZC_TYPE_{t}"]) for t in ("BF16", "FP16", "FP32")]


def test_sizes():
    f = _tensors.fn
    assert f("zc_fp8_column_blocks")(1000, 4) == 7 + 4
    assert f("zc_fp8_column_blocks")(3, 10) == 3
    assert f("zc_fp8_column_blocks")(0, 10) == 0
    assert f("zc_fp8_column_blocks")(100, 0) == 0 == f("zc_fp8_column_blocks")(100, 1025)
    assert f("zc_moe_sort_workspace")(100, 8) == 0  # small calls need none
    assert f("zc_moe_sort_workspace")(100000, 8) >= 9 * 4
    assert f("zc_fp8_matmul_workspace")(8, 1, 4096, 7168) > 0 == f("zc_fp8_matmul_workspace")(0, 1, 4096, 7168)
    assert f("zc_fp8_matmul_workspace")(4096, 1, 4096, 7168) == 0 == f("zc_fp8_matmul_workspace")(8, 0, 4096, 7168)
    assert f("zc_fp8_matmul_workspace")(8, 1, 4096, 2048) == 0  # short sums need none
    assert f("zc_moe_sort_workspace")((1 << 30) + 1, 8) == 0 == f("zc_moe_sort_workspace")(10, 0)


def refused(name, args, changes):
    fn = _tensors.fn(name)
    for at, value, code in changes:
        bad = list(args)
        bad[at] = value
        assert fn(*bad) == code, (name, at, value)


INV, MIS = zc.ZC_ERR_INVALID_ARG, zc.ZC_ERR_MISALIGNED


def test_sort_and_dispatch_refuse():
    refused("zc_moe_sort", [A, 4, 10, 2, 4, B, C, D, 0],
            [(0, 0, INV), (1, 2, INV), (3, 0, INV), (3, 65, INV), (4, 0, INV), (4, 1025, INV), (5, 0, INV), (6, 0, INV),
             (0, A + 2, MIS), (5, B + 2, MIS), (6, C + 1, MIS), (7, D + 8, MIS), (5, A + 4, INV),
             (6, B + 8, INV), (2, 1 << 30, INV)])
    refused("zc_moe_sort", [A, 4, 10000, 2, 4, B, C, D, 0], [(7, 0, INV)])  # many slots: a workspace
    refused("zc_moe_dispatch", [A, 64, 0, B, 4, 10000, 2, 4, 64, C, 64, D, E, F, 0], [(13, 0, INV)])
    refused("zc_moe_dispatch", [A, 64, 0, B, 4, 10, 2, 4, 64, C, 64, D, E, F, 0],
            [(0, 0, INV), (1, 63, INV), (2, 3, INV), (2, -1, INV), (3, 0, INV), (4, 3, INV), (6, 0, INV), (7, 0, INV),
             (8, 0, INV), (9, 0, INV), (10, 63, INV), (11, 0, INV), (12, 0, INV), (0, A + 1, MIS),
             (9, C + 1, MIS), (9, A + 128, INV), (9, B, INV), (9, D, INV)])


def test_combine_refuses():
    refused("zc_moe_combine", [A, 64, 0, B, C, D, 10, 2, 4, 64, E, 64, 0],
            [(0, 0, INV), (1, 63, INV), (2, 3, INV), (4, 0, INV), (5, 0, INV), (7, 0, INV), (8, 0, INV), (9, 0, INV),
             (10, 0, INV), (11, 1, INV), (0, A + 1, MIS), (3, B + 2, MIS), (4, C + 2, MIS), (5, D + 2, MIS),
             (10, A + 64, INV), (10, B, INV)])
    refused("zc_moe_combine_grad", [A, 64, 0, 64, 0, B, C, D, 10, 2, 4, 64, E, 64, F, 0], [(2, 0, INV)])
    refused("zc_moe_combine_grad", [A, 64, B, 64, 0, C, D, E, 10, 2, 4, 64, F, 64, F * 2, 0],
            [(0, 0, INV), (1, 1, INV), (3, 1, INV), (4, 7, INV), (5, 0, INV), (6, 0, INV), (7, 0, INV), (9, 99, INV),
             (10, 0, INV), (11, 0, INV), (12, 0, INV), (13, 1, INV), (14, 0, INV), (0, A + 1, MIS), (14, F * 2 + 2, MIS),
             (12, A, INV), (12, B, INV), (14, F, INV)])


def test_quantize_refuses():
    refused("zc_fp8_quantize", [A, 256, 0, 10, 256, 0, B, C, 0],
            [(0, 0, INV), (1, 255, INV), (2, 3, INV), (4, 0, INV), (5, 2, INV), (6, 0, INV), (7, 0, INV), (0, A + 1, MIS),
             (6, B + 8, MIS), (7, C + 2, MIS), (6, A, INV), (7, B, INV), (4, (1 << 20) + 1, INV), (3, 1 << 31, INV)])
    refused("zc_fp8_scale_values", [A, 64, B, 0],
            [(0, 0, INV), (1, 1 << 31, INV), (2, 0, INV), (0, A + 1, MIS), (2, B + 8, MIS), (2, A + 240, INV)])
    refused("zc_fp8_quantize_columns", [A, 256, 0, 10, 256, 3, B, 0, C, D, E, 0],
            [(0, 0, INV), (1, 255, INV), (5, 0, INV), (5, 1025, INV), (6, 0, INV), (7, 2, INV), (8, 0, INV), (9, 0, INV),
             (10, 0, INV), (8, C + 8, MIS), (8, A, INV), (10, C, INV)])
    refused("zc_fp8_quantize_weight", [A, 0, 2, 64, 128, 0, B, C, D, E, 0],
            [(0, 0, INV), (1, 9, INV), (2, 0, INV), (3, 0, INV), (4, 0, INV), (5, 2, INV), (6, 0, INV), (7, 0, INV),
             (8, 0, INV), (9, 0, INV), (6, B + 1, MIS), (8, B, INV)])


def test_products_refuse():
    refused("zc_fp8_matmul", [A, B, 0, 10, C, D, 0, 2, 64, 128, E, F, 64, 0, F * 2, 0],
            [(0, 0, INV), (1, 0, INV), (2, 2, INV), (4, 0, INV), (5, 0, INV), (6, -1, INV), (7, 0, INV), (8, 0, INV),
             (9, 0, INV), (10, 0, INV), (11, 0, INV), (12, 63, INV), (13, 1, INV), (0, A + 16, MIS), (4, C + 64, MIS),
             (1, B + 2, MIS), (11, F + 1, MIS), (11, A, INV), (11, C, INV)])
    refused("zc_fp8_matmul", [A, B, 0, 10, C, D, 0, 2, 64, 8192, E, F, 64, 0, F * 2, 0],  # long sums: a workspace
            [(14, 0, INV), (14, F * 2 + 4, MIS), (14, F, INV)])
    refused("zc_fp8_weight_grad", [A, B, 0, C, D, 0, 4, 2, 64, 128, E, F, 0, 0],
            [(0, 0, INV), (1, 0, INV), (2, 2, INV), (3, 0, INV), (5, 5, INV), (7, 0, INV), (8, 0, INV), (9, 0, INV),
             (10, 0, INV), (11, 0, INV), (12, 1, INV), (0, A + 16, MIS), (10, E + 2, MIS), (11, C, INV)])


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="checks the no-GPU failure path")
def test_no_gpu_fails_loudly():
    assert _tensors.fn("zc_moe_sort")(A, 4, 10, 2, 4, B, C, D, 0) == zc.ZC_ERR_CUDA
    assert _tensors.fn("zc_moe_combine")(A, 64, 0, B, C, D, 10, 2, 4, 64, E, 64, 0) == zc.ZC_ERR_CUDA
    assert _tensors.fn("zc_fp8_quantize")(A, 256, 0, 10, 256, 0, B, C, 0) == zc.ZC_ERR_CUDA
    assert _tensors.fn("zc_fp8_matmul")(A, B, 0, 10, C, D, 0, 2, 64, 128, E, F, 64, 0, F * 2, 0) == zc.ZC_ERR_CUDA
    import torch

    from lossless_bf16_compression_gb300 import fp8, moe
    with pytest.raises(TypeError):
        moe.sort(torch.zeros((2, 2), dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        fp8.quantize(torch.zeros((2, 2)))


def test_native_calls_refuse():
    """The calls on tensors, with arguments that never reach the library."""
    torch = pytest.importorskip("torch")
    native, x = _tensors.native, torch.zeros((4, 8))
    for name, args in (("sort", ()), ("sort", (x.int(), 4, 1)), ("sort", (x.int(), 4)), ("sort", ([[0]], 4)), ("sort", (None, 4)),
                       ("dispatch", (x, x.int(), 4)), ("combine", (x, None, x.int(), x.int())), ("combine", (x,)),
                       ("combine_grad", (x,) * 5), ("quantize", (x, 0)), ("quantize", ("x", 0)), ("quantize_columns", (x, None, 0)),
                       ("quantize_weight", (x, 0, True)), ("scale_values", (x.byte(),)), ("values", (3, 0, 8)),
                       ("matmul", (x.byte(), x.byte(), 0, 8) * 2 + (None, 0)), ("weight_grad", (x.byte(),)), ("bind", ())):
        with pytest.raises(TypeError):
            getattr(native, name)(*args)
    q = native.values(torch.arange(8, dtype=torch.uint8).view(2, 4), 0, 3)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (2, 3) and q.stride() == (4, 1)
