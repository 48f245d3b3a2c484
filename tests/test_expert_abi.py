"""Entry points of include/zc_moe.h without a GPU: the test hooks refuse what the calls they stand for refuse."""
import os

import pytest

from lossless_bf16_compression_gb300 import binding as zc
from lossless_bf16_compression_gb300 import build as zbuild

pytest.importorskip("torch")
from lossless_bf16_compression_gb300 import _tensors  # noqa: E402

A = 1 << 30  # aligned fake addresses, far apart; never dereferenced by calls that are refused
B, C, D, E, F = (A * i for i in range(2, 7))
INV, MIS = zc.ZC_ERR_INVALID_ARG, zc.ZC_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def _built():
    zbuild.build()


@pytest.mark.parametrize("name,args,changes", [
    ("zc_fp8_matmul_stall_test", [A, B, 0, 10, C, D, 0, 2, 64, 128, E, F, 64, 0, F * 2, 0, 0, 1000],
     [(0, 0, INV), (2, 2, INV), (7, 0, INV), (8, 0, INV), (10, 0, INV), (12, 63, INV), (13, 1, INV), (0, A + 16, MIS),
      (11, A, INV)]),
    ("zc_fp8_weight_grad_stall_test", [A, B, 0, C, D, 0, 4, 2, 64, 128, E, F, 0, 0, 0, 1000],
     [(0, 0, INV), (2, 2, INV), (7, 0, INV), (10, 0, INV), (12, 1, INV), (0, A + 16, MIS), (11, C, INV)]),
])
def test_stall_hooks_refuse(name, args, changes):
    fn = _tensors.fn(name)
    for at, value, code in changes:
        bad = list(args)
        bad[at] = value
        assert fn(*bad) == code, (at, value)
    if not os.path.exists("/dev/nvidia0"):
        assert fn(*args) == zc.ZC_ERR_CUDA  # valid arguments reach the runtime, which has no device


def test_weight_grad_takes_what_quantize_columns_makes():
    """The most blocks that quantize_columns fills, of the most rows in the most groups, and not one more."""
    rows, groups, far = 0x7FFFFFFF - 131072, 1024, 1 << 40
    most = _tensors.fn("zc_fp8_column_blocks")(rows, groups)
    assert most == rows // 128 + groups and _tensors.fn("zc_fp8_column_blocks")(rows + 1, groups) == 0
    fn = _tensors.fn("zc_fp8_weight_grad")

    def rc(capacity):
        return fn(far, 2 * far, 0, 3 * far, 4 * far, 0, capacity, groups, 1, 1, 5 * far, 6 * far, 2, 0)

    assert rc(most + 1) == INV
    if not os.path.exists("/dev/nvidia0"):
        assert rc(most) == zc.ZC_ERR_CUDA == rc(rows // 128 + 1)


def test_kernel_ids_match_the_header():
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    found = {}
    for name in ("zc.h", "zc_moe.h"):
        found |= dict(re.findall(r"^#define\s+(ZC_KERNEL_\w+)\s+(\d+)", open(os.path.join(root, "include", name)).read(), flags=re.M))
    assert len(set(found.values())) == len(found) == 18
    for name, value in found.items():
        assert getattr(zc, name) == int(value), name


def test_a_checkout_that_is_not_built_says_so_on_first_use():
    """moe and fp8 import without the extension module (a checkout that is not built yet); their first call says what is
    missing."""
    import subprocess
    import sys

    code = """
import sys
name = "lossless_bf16_compression_gb300._experts"
sys.modules[name] = None  # as if it were not there
import torch
from lossless_bf16_compression_gb300 import fp8, moe
for call in (lambda: moe.sort(torch.zeros((2, 2), dtype=torch.int32), 4), lambda: fp8.quantize(torch.zeros((2, 2)))) * 2:
    try:
        call()
    except ImportError as e:
        assert "build" in str(e), e
    else:
        raise SystemExit("no error")
del sys.modules[name]
try:
    moe.sort(torch.zeros((2, 2), dtype=torch.int32), 4)  # built by now: refused for the tensor
except TypeError:
    print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr
