"""Build the retrieval library in-tree: nvcc -> hash_hierarchical_top_b200/libhhr.so (sm_100a),
and the Python marshalling module beside it: g++ -> hash_hierarchical_top_b200/_binding.so.

Run ``python -m hash_hierarchical_top_b200.build`` (or call ``build()``). The
library is a single CUDA translation unit; nvcc cross-compiles it without a GPU.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libhhr.so")
BINDING = os.path.join(HERE, "_binding.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh"))] + [os.path.join(ROOT, "include", "hhr.h")]


def _fresh(target, srcs):
    return os.path.exists(target) and all(os.path.getmtime(s) <= os.path.getmtime(target)
                                          for s in srcs)


def binding_tag() -> str:
    """What _binding.so is built against: it uses torch's C++ types and Python's C API, which hold
    for one release each."""
    import torch
    return f"hhr binding for torch {torch.__version__}, {sys.implementation.cache_tag}"


def binding_matches(path: str = BINDING) -> bool:
    """Whether the module at `path` was built against the installed torch and Python (the tag is one
    of its strings, so that it need not be loaded to be asked)."""
    with open(path, "rb") as f:
        return binding_tag().encode() + b"\0" in f.read()


def build_binding(force: bool = False):
    """Start compiling _binding.so (against the installed torch's headers) if it is missing, older
    than its sources or built against another torch or Python; returns the process, or None."""
    src = os.path.join(CSRC, "binding.cpp")
    if (not force and _fresh(BINDING, [src, os.path.join(ROOT, "include", "hhr.h")])
            and binding_matches()):
        return None
    import torch
    from torch.utils.cpp_extension import CUDA_HOME, include_paths
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = include_paths() + [sysconfig.get_paths()["include"],
                             os.path.join(CUDA_HOME or "/usr/local/cuda", "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DHHR_BUILT_FOR="{binding_tag()}"',
           *(f"-I{i}" for i in inc), "-o", BINDING + ".tmp", src, f"-L{libs}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return subprocess.Popen(cmd)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libhhr.so and _binding.so where they are missing or out of date; return the
    library's path."""
    binding = build_binding(force)
    try:
        return _build_lib(force, verbose)
    finally:
        if binding is not None:
            if binding.wait() != 0:
                raise RuntimeError("building _binding.so failed")
            os.replace(BINDING + ".tmp", BINDING)


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and _fresh(LIB, sources()):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    if os.path.exists("/usr/local/cuda/bin/nvcc") and nvcc == "nvcc":
        nvcc = "/usr/local/cuda/bin/nvcc"
    tmp = LIB + ".tmp"
    cmd = [nvcc, *NVCC_FLAGS, "-o", tmp, os.path.join(CSRC, "hhr_api.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
