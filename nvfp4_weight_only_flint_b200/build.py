"""Build libflint_moe.so in-tree with nvcc for sm_100a (B200), and the Python marshalling module beside it with g++."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SO = os.path.join(PKG, "libflint_moe.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
OBJ_DIR = os.path.join(PKG, "_build")
MARSHAL_FOR = os.path.join(OBJ_DIR, "marshal.txt")  # what _marshal.so was built for
# translation units, compiled in parallel and linked into one shared library
SOURCES = ["flint_moe.cu", "tok1.cu", "tokn.cu", "lmhead.cu", "attn.cu", "attn_decode.cu", "ep.cu",
           "paged_kv.cu", "paged_attn.cu", "paged_decode.cu", "paged_chunk.cu", "sample.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


def _marshal_built_for() -> str:
    """The interpreter and the torch that the extension module is compiled for (read without importing torch)."""
    from importlib.metadata import version
    return f"python {sys.version} torch {version('torch')}"


def _marshal_is_current() -> bool:
    header = os.path.join(INCLUDE, "flint_moe.h")
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_FOR):
        return False
    with open(MARSHAL_FOR) as f:
        if f.read() != _marshal_built_for():
            return False
    return all(os.path.getmtime(f) <= os.path.getmtime(MARSHAL) for f in (MARSHAL_SRC, header))


def _build_marshal(force: bool, verbose: bool) -> None:
    """The extension module needs torch's headers and links against torch and libflint_moe.so (found beside it)."""
    if not force and _marshal_is_current():
        return
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}", *[f"-I{d}" for d in include_paths()], MARSHAL_SRC,
           "-o", tmp, *[f"-L{d}" for d in library_paths()], f"-L{PKG}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
           "-ltorch_python", "-l:libflint_moe.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, MARSHAL)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(MARSHAL_FOR, "w") as f:
        f.write(_marshal_built_for())


def build(force: bool = False, verbose: bool = False) -> str:
    so = _build_library(force, verbose)
    _build_marshal(force, verbose)
    return so


def _build_library(force: bool, verbose: bool) -> str:
    if not force and os.path.exists(SO):
        so_time = os.path.getmtime(SO)
        if all(os.path.getmtime(f) <= so_time for f in _inputs()):
            return SO
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ_DIR, exist_ok=True)
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + f".{os.getpid()}.o")
        cmd = [nvcc, *NVCC_FLAGS, f"-I{INCLUDE}", "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        objs.append(obj)
        procs.append(subprocess.Popen(cmd))
    failed = [p.wait() for p in procs]
    if any(failed):
        for o in objs:
            if os.path.exists(o):
                os.unlink(o)
        raise subprocess.CalledProcessError(max(failed), "nvcc")
    tmp = SO + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    for o in objs:
        os.unlink(o)
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
