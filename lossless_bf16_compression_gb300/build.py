"""Build the sm_103a CUDA library ``libzc.so`` in-tree with nvcc (no torch, no cmake), and with g++ the
extension module ``_experts`` (``moe`` and ``fp8``'s calls on torch tensors; built where torch is installed).

Each translation unit compiles in parallel into ``_build/``; the shared object links the
CUDA runtime statically, so it loads into any process that has the NVIDIA driver.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libzc.so")
MODULE_PATH = os.path.join(PKG, "_experts.so")
MODULE_SOURCE = os.path.join(CSRC, "experts", "ex_torch.cpp")
SOURCES = ["zc_api.cu", "zc_stats.cu", "zc_encode.cu", "zc_decode.cu", "zc_static.cu", "zc_small.cu", "zc_fused.cu",
           "experts/ex_api.cu", "experts/ex_sort.cu", "experts/ex_rows.cu", "experts/ex_quantize.cu",
           "experts/ex_matmul.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libzc.so")


def _inputs() -> list[str]:
    files = [os.path.join(d, f) for top in (CSRC, INCLUDE) for d, _, names in os.walk(top) for f in names]
    torch = _torch()
    return files + [os.path.abspath(__file__)] + ([os.path.join(torch, "version.py")] if torch else [])


def _torch() -> str | None:
    """Where torch is installed (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _build_module(verbose: bool) -> None:
    torch = _torch()
    if torch is None:
        return
    tmp = MODULE_PATH + f".tmp{os.getpid()}"
    headers = os.path.join(torch, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-o", tmp, MODULE_SOURCE, f"-I{INCLUDE}",
           f"-isystem{headers}", f"-isystem{headers}/torch/csrc/api/include", f"-isystem{cuda}",
           f"-isystem{sysconfig.get_paths()['include']}", f"-L{os.path.join(torch, 'lib')}", "-ltorch_python",
           "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MODULE_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE_PATH)


def up_to_date() -> bool:
    made = [LIB_PATH] + ([MODULE_PATH] if _torch() else [])
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link libzc.so for sm_103a; return its path."""
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace("/", "_").replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(_build_module, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        module.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
