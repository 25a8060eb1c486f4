"""Build step of the package: compiles the CUDA sources into ``libmsa.so`` in-tree.

``python -m block_sparse_gqa_03_b200.build`` (or ``__graft_entry__.build()``)
runs nvcc once per source for sm_100a and links a shared library next to this
file.  The library exports only the C ABI of ``include/msa.h``.  The binding's
marshalling extension ``_marshal.so`` is compiled next to it.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
MARSHAL = os.path.join(HERE, "_marshal.so")  # Python extension: argument checks of the q8 calls
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["msa_api.cu", "index_scores.cu", "index_scores_tc.cu", "topk.cu", "sparse_attn.cu",
           "sparse_attn_kv.cu", "append_kv.cu", "shard.cu", "kv_q8.cu", "index_scores_q8.cu",
           "sparse_attn_q8.cu"]
HEADERS = ["attn_common.cuh", "common.cuh", "kernels.h", "q8.cuh", "sm100.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "msa.h")]
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [path] + hdrs):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", path, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp, "-lcudart_static",
               "-ldl", "-lrt", "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_marshal(force, verbose)
    return LIB


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compiles the marshalling extension against this interpreter's and torch's headers."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "marshal.cpp")
    if force or _stale(MARSHAL, [src, os.path.join(ROOT, "include", "msa.h")]):
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        tmp = MARSHAL + ".tmp%d" % os.getpid()
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
               "-fvisibility=hidden", "-I" + inc,
               "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
               "-I" + sysconfig.get_paths()["include"], src, "-o", tmp, "-L" + lib,
               "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
