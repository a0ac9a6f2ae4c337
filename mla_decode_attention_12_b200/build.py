"""Builds the C-ABI shared library ``_mla_decode.so`` in-tree with nvcc for sm_100a, and the
PyTorch binding ``_mla_torch.so`` beside it.

Usage: ``python -m mla_decode_attention_12_b200.build`` (or call :func:`build`).
The CUDA runtime is linked statically, so the library needs only the NVIDIA
driver at run time.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "_mla_decode.so")
BINDING = os.path.join(HERE, "_mla_torch.so")
BINDING_STAMP = BINDING + ".built_with"  # the torch and Python that it was built with
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
HEADER = os.path.join(ROOT, "include", "mla_decode.h")
SOURCES = [os.path.join(CSRC, f) for f in ("mla_decode.cu", "cache_ops.cu", "select_pages.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("host_util.cuh", "ptx.cuh", "scheduler.cuh")] + [HEADER]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date(out: str = LIB, deps=None) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in (DEPS if deps is None else deps))


def binding_stamp() -> str:
    """What a binding works with alone: torch's version and C++ ABI, and Python's ABI."""
    import torch

    return f"torch {torch.__version__} cxx11_abi {int(torch.compiled_with_cxx11_abi())} {sysconfig.get_config_var('SOABI')}\n"


def binding_up_to_date() -> bool:
    if not up_to_date(BINDING, [BINDING_SOURCE, HEADER]):
        return False
    try:
        with open(BINDING_STAMP, encoding="utf-8") as f:
            return f.read() == binding_stamp()
    except OSError:
        return False


def build(force: bool = False, verbose: bool = False, extra=(), out: str = LIB) -> str:
    """Compile the library if any source is newer than it; returns its path.

    ``extra`` adds nvcc flags and ``out`` names another file: instrumented or test-only
    builds of the same sources (``-DMLA_TIMELINE``, ``-DMLA_TEST_WITHHOLD_K_PAGE=n``) go
    to their own files, never to the product library's.  The product build includes the
    PyTorch binding; where that does not build (no torch headers, say), the library does all the
    same, and the error is raised after it."""
    todo = []
    tmp = out + f".tmp{os.getpid()}"
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor() as pool:
        if force or not up_to_date(out):
            objs = [os.path.join(objects, os.path.basename(src) + ".o") for src in SOURCES]
            flags = [f for f in NVCC_FLAGS if f != "-shared"]
            todo = [pool.submit(_run, [nvcc(), *flags, *extra, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src], verbose)
                    for src, obj in zip(SOURCES, objs)]
        binding = compiled = None
        if out == LIB:
            binding = os.path.join(objects, "binding.o")
            compiled = pool.submit(_compile_binding, binding, verbose, force)
        for t in todo:
            t.result()
        if todo:
            _run([nvcc(), *NVCC_FLAGS, "-o", tmp, *objs], verbose)
            os.replace(tmp, out)
        if compiled is not None and compiled.result():
            _link_binding(binding, verbose)
    return out


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)


def _torch_dir() -> str:
    import torch

    return os.path.dirname(torch.__file__)


def _compile_binding(obj: str, verbose: bool, force: bool) -> bool:
    """Compiles the binding unless it is up to date; whether it did."""
    if not force and binding_up_to_date():
        return False
    import torch

    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          *(f for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda, sysconfig.get_paths()["include"])
            for f in ("-isystem", d)), "-c", "-o", obj, BINDING_SOURCE], verbose)
    return True


def _link_binding(obj: str, verbose: bool) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:_mla_decode.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"], verbose)
    os.replace(tmp, BINDING)
    with open(tmp, "w", encoding="utf-8") as f:
        f.write(binding_stamp())
    os.replace(tmp, BINDING_STAMP)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
