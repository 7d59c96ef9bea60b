"""Build libsparse_attn.so in-tree for sm_100a with nvcc (one shared
library, C ABI, no torch types), and beside it _paged, the Python module that
marshals the paged cache's calls (host C++ on torch's headers).
Usage: python -m sparse_graph_causal_b200.build"""
from __future__ import annotations

import importlib.metadata
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsparse_attn.so")
OBJ = os.path.join(HERE, "_build")
BIND = os.path.join(HERE, "_paged" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _text(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def build(verbose: bool = False, jobs: int = 8) -> str:
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(HERE, "..", "include", "sparse_attn.h"))
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        if _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd))
            procs.append((src, subprocess.Popen(cmd)))
        while len([p for _, p in procs if p.poll() is None]) >= jobs:
            procs[0][1].wait()
    for src, p in procs:
        if p.wait() != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    if _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """The module holds torch's C++ interface of the version that it is built with: it is built
    again for another one (kept beside the objects), and refuses to load next to one."""
    src = os.path.join(CSRC, "paged_py.cpp")
    stamp = os.path.join(OBJ, os.path.basename(BIND) + ".torch")
    version = importlib.metadata.version("torch")
    if _stale(BIND, [src, os.path.join(HERE, "..", "include", "sparse_attn.h")]) \
            or _text(stamp) != version:
        import torch
        from torch.utils.cpp_extension import include_paths, library_paths
        cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
               f'-DSA_TORCH_VERSION="{torch.__version__}"']
        cmd += [f"-I{p}" for p in (*include_paths(), cuda, sysconfig.get_paths()["include"])]
        cmd += [src, "-o", BIND, *(f"-L{p}" for p in library_paths()), "-lc10", "-lc10_cuda",
                "-ltorch_cpu", "-ltorch_python", f"-L{HERE}", f"-l:{os.path.basename(LIB)}",
                "-Wl,-rpath,$ORIGIN"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.makedirs(OBJ, exist_ok=True)
        with open(stamp, "w") as f:
            f.write(version)
    return BIND


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
