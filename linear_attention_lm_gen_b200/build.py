"""Build the JetBlock CUDA library (libjet.so) in-tree for sm_100a with nvcc, and
the fast path of its Python binding (_bind.so) with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libjet.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def sources():
    out = []
    for d, _, files in os.walk(CSRC):
        out += [os.path.join(d, f) for f in files if f.endswith((".cu", ".cuh", ".h"))]
    out.append(os.path.join(INCLUDE, "jet.h"))
    return out


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, out: str = LIB) -> str:
    """Compile csrc/jet_api.cu (which includes every kernel) into libjet.so
    (or, for a test build with extra defines, into `out`)."""
    if out == LIB:
        build_bind(force, verbose)
    if not force and os.path.exists(out):
        mt = os.path.getmtime(out)
        if all(os.path.getmtime(s) <= mt for s in sources()):
            return out
    cmd = [NVCC, *FLAGS, *(extra or []), "-I", INCLUDE, "-I", CSRC,
           "-o", out + ".tmp", os.path.join(CSRC, "jet_api.cu")]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def bind_abi() -> str:
    """What _bind.so is built against: it calls torch's C++ interface and CPython's own."""
    import torch
    return f"torch {torch.__version__} {sys.implementation.cache_tag}"


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/bind.cpp, a CPython module on torch's C++ interface, into
    _bind.so. _bind.abi beside it says for which torch and Python."""
    header, stamp, abi = os.path.join(INCLUDE, "jet.h"), os.path.splitext(BIND)[0] + ".abi", bind_abi()
    if not force and os.path.exists(BIND) and os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == abi
        if same and all(os.path.getmtime(s) <= os.path.getmtime(BIND) for s in (BIND_SRC, header)):
            return BIND
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DJET_BIND_ABI="{abi}"',
           *[f"-I{d}" for d in inc], BIND_SRC, "-o",
           BIND + ".tmp", "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(BIND + ".tmp", BIND)
    with open(stamp, "w") as f:
        f.write(abi)
    return BIND


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
