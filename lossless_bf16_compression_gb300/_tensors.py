"""What the tensor-level calls of ``moe`` and ``fp8`` share: argument checks, streams, the library's calls."""
from __future__ import annotations

import contextlib
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
}

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_EXPERTS = 1024
MAX_K = 64

_fns: dict = {}


def fn(name):
    """An entry point of the library with its argument types set; raises when the library is not built."""
    f = _fns.get(name)
    if f is None:
        handle = binding.lib()
        f = getattr(handle, name)
        f.restype, f.argtypes = SIGNATURES[name]
        _fns[name] = f
    return f


def call(name, *args):
    rc = (_fns.get(name) or fn(name))(*args)
    if rc != binding.ZC_OK:
        raise binding.ZcError(rc, name)


def check(ok, what):
    if not ok:
        raise ValueError(what)


def on_device(name, t, device, dtypes=None, dim=None):
    """Checks for a CUDA tensor of device number `device` (None: the current one), of one of `dtypes`, with `dim`
    dimensions; returns the device number."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {', '.join(str(d) for d in dtypes)}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {tuple(t.shape)}")
    if device is None:
        device = torch._C._cuda_getDevice()
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return device


def rows_of(t):
    """(tensor, pitch): `t` as rows of contiguous values a pitch apart (copied when it is not laid out so)."""
    rows, cols = t.shape
    pitch, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and pitch < cols):
        t, pitch = t.contiguous(), cols
    return t, (pitch if rows > 1 else cols)


def on(stream, used, f, *args):
    """f(*args) with `stream` (None: the current one) as the current stream, so that what it allocates is the
    stream's.  The tensors `used` there are kept from reuse until the stream has passed the call."""
    if stream is None:
        return f(*args)
    for t in used:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return f(*args)


current = torch._C._cuda_getCurrentRawStream  # (device) -> the handle of its current stream
