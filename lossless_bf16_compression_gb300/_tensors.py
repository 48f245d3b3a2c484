"""What the tensor-level calls of ``moe`` and ``fp8`` share: the native calls, streams, the C entry points."""
from __future__ import annotations

import ctypes

import torch

from . import binding

_P, _N, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int

# (restype, argtypes) of every entry point of zc_moe.h.
SIGNATURES = {
    "zc_moe_sort_workspace": (_N, [_N, _I]),
    "zc_moe_sort": (_I, [_P, _I, _N, _I, _I, _P, _P, _P, _P]),
    "zc_moe_dispatch": (_I, [_P, _N, _I, _P, _I, _N, _I, _I, _N, _P, _N, _P, _P, _P, _P]),
    "zc_moe_combine": (_I, [_P, _N, _I, _P, _P, _P, _N, _I, _I, _N, _P, _N, _P]),
    "zc_moe_combine_grad": (_I, [_P, _N, _P, _N, _I, _P, _P, _P, _N, _I, _I, _N, _P, _N, _P, _P]),
    "zc_fp8_quantize": (_I, [_P, _N, _I, _N, _N, _I, _P, _P, _P]),
    "zc_fp8_scale_values": (_I, [_P, _N, _P, _P]),
    "zc_fp8_column_blocks": (_N, [_N, _I]),
    "zc_fp8_quantize_columns": (_I, [_P, _N, _I, _N, _N, _I, _P, _I, _P, _P, _P, _P]),
    "zc_fp8_quantize_weight": (_I, [_P, _I, _I, _N, _N, _I, _P, _P, _P, _P, _P]),
    "zc_fp8_matmul_workspace": (_N, [_N, _I, _N, _N]),
    "zc_fp8_matmul": (_I, [_P, _P, _I, _N, _P, _P, _I, _I, _N, _N, _P, _P, _N, _I, _P, _P]),
    "zc_fp8_weight_grad": (_I, [_P, _P, _I, _P, _P, _I, _N, _I, _N, _N, _P, _P, _I, _P]),
    "zc_fp8_matmul_stall_test": (_I, [_P, _P, _I, _N, _P, _P, _I, _I, _N, _N, _P, _P, _N, _I, _P, _P, _I, _I]),
    "zc_fp8_weight_grad_stall_test": (_I, [_P, _P, _I, _P, _P, _I, _N, _I, _N, _N, _P, _P, _I, _P, _I, _I]),
}

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_EXPERTS = 1024
MAX_K = 64


def fn(name):
    """An entry point of the library with its argument types set, for callers that have addresses instead of
    tensors; raises when the library is not built."""
    f = getattr(binding.lib(), name)
    f.restype, f.argtypes = SIGNATURES[name]
    return f


def _load():
    try:
        from . import _experts
    except ImportError as e:
        raise ImportError("the extension module _experts is missing or was built for another torch: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')") from e
    _experts.bind(binding.lib()._handle, binding.ZcError)
    return _experts


class _NotBuilt:
    """Stands for the extension module in a checkout that is not built yet: a call loads it, or says what is missing."""

    def __getattr__(self, name):
        module = _load()
        self.__dict__.update((k, v) for k, v in vars(module).items() if not k.startswith("__"))
        return getattr(module, name)


try:
    native = _load()  # the calls on tensors: checks, outputs, launch, on the current device and stream
except (ImportError, RuntimeError):
    native = _NotBuilt()


def on(stream, used, f, *args):
    """f(*args) with `stream` (None: the current one) as the current stream, so that what it allocates is the
    stream's.  The tensors `used` there are kept from reuse until the stream has passed the call."""
    if stream is None:
        return f(*args)
    for t in used:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return f(*args)
