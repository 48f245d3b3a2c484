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
