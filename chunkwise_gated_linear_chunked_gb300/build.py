"""Build libgla.so in-tree (``chunkwise_gated_linear_chunked_gb300/_build/``) with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit compiles in parallel to an object file; nvcc then links them into one
shared library with the C ABI of ``include/gla.h``.  Beside it the host compiler builds ``_calls``, a small CPython
module against torch's headers that shortens the binding's usual calls (``csrc/torch_calls.cpp``).  No torch
extension machinery is involved.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgla.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgla")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "gla.h"), os.path.abspath(__file__)]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in _deps())


def calls_lib() -> str:
    """The _calls module's file, which belongs to one version of torch."""
    import torch
    return os.path.join(BUILD, f"_calls-{torch.__version__}.so")


def calls_stale() -> bool:
    lib = calls_lib()
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in (CALLS_SRC, os.path.join(ROOT, "include", "gla.h"),
                                                 os.path.abspath(__file__)))


def build_calls() -> None:
    """Compile and link the _calls module against libgla.so (which lies beside it) and torch.  The binding works without it
    (each call of the layer operators then takes some ten microseconds more on the host), so a failure is a warning."""
    try:
        _build_calls()
    except (OSError, RuntimeError) as e:
        if os.path.exists(calls_lib()):   # of an earlier state of the library
            os.remove(calls_lib())
        warnings.warn(f"_calls was not built, the binding goes without: {e}", RuntimeWarning, stacklevel=2)


def _build_calls() -> None:
    import torch
    home, lib = os.path.dirname(torch.__file__), calls_lib()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           CALLS_SRC, "-o", tmp, "-L", BUILD, "-l:libgla.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda",
           "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {CALLS_SRC}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not stale():
        if calls_stale():
            build_calls()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include")]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            print(res.stdout + res.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".{os.getpid()}.tmp"
    res = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    build_calls()
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
