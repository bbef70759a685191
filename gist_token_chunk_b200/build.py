"""Build step for libssa.so (sm_100a) -- run by ``__graft_entry__.build()``.

Compiles the CUDA kernels and the C ABI with nvcc into
``gist_token_chunk_b200/libssa.so`` (in-tree, static CUDA runtime), and the
native part of the Python binding with g++ into ``binding_path()``.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssa.so")
SOURCES = ["ssa_kernels.cu", "ssa_api.cpp", "ssa_prefill.cu", "ssa_q8.cu", "ssa_rope.cu"]
HEADERS = ["ssa_device.cuh", "ssa_fused.cuh", "ssa_generic.cuh", "ssa_internal.h", "ssa_pipe.cuh",
           "ssa_q8.h", "ssa_q8_cache.cuh", "ssa_q8_decode.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


BINDING_SOURCE = os.path.join(CSRC, "py_cache.cpp")


def binding_path() -> str:
    """The binding for this Python and torch, whose binary interfaces it is tied to."""
    import torch

    tag = f"{sys.implementation.cache_tag}-torch-{torch.__version__}"
    return os.path.join(HERE, f"_cache.{tag}.so")


def _start_binding(force: bool):
    """Starts compiling the binding when it is out of date; (process, temporary
    file) or None."""
    import sysconfig

    import torch

    path = binding_path()
    deps = [BINDING_SOURCE, os.path.join(ROOT, "include", "ssa.h"), os.path.abspath(__file__)]
    if (not force and os.path.exists(path)
            and os.path.getmtime(path) >= max(os.path.getmtime(d) for d in deps)):
        return None
    base = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-o", tmp,
           BINDING_SOURCE, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for d in include for x in ("-isystem", d)]
    cmd += ["-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return subprocess.Popen(cmd), tmp


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "ssa.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False, extra=(), out: str = LIB) -> str:
    """Compile libssa.so; ``extra`` nvcc flags (e.g. -DSSA_TRACE) and another
    ``out`` path give instrumented variants without touching the product."""
    binding = _start_binding(force) if out == LIB else None
    try:
        if out != LIB or force or _stale():
            _build_library(verbose, extra, out)
    finally:
        if binding is not None:
            failed = binding[0].wait()
    if binding is not None:
        if failed:
            raise subprocess.CalledProcessError(failed, binding[0].args)
        os.replace(binding[1], binding_path())
    return out


def _build_library(verbose: bool, extra, out: str) -> None:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC,-O3,-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
           "-o", tmp, *[os.path.join(CSRC, f) for f in SOURCES], *extra]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
