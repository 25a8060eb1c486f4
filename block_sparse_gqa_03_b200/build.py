"""Build step of the package: compiles the CUDA sources into ``libmsa.so`` in-tree.

``python -m block_sparse_gqa_03_b200.build`` (or ``__graft_entry__.build()``)
runs nvcc once per source for sm_100a and links a shared library next to this
file.  The library exports only the C ABI of ``include/msa.h``.  The binding's
marshalling extension ``_marshal.<torch and Python version>.so`` is compiled next to it.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmsa.so")
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


def marshal_path() -> str:
    """The marshalling extension (argument checks of the 8-bit calls).  It is bound to the
    C++ ABI of the torch and the Python it was compiled for, which its name holds: after a
    change of either the old file is not found, instead of being loaded."""
    import torch

    return os.path.join(HERE, "_marshal.torch%s%s" % (torch.__version__,
                                                      sysconfig.get_config_var("EXT_SUFFIX")))


def build_marshal(force: bool = False, verbose: bool = False) -> str | None:
    """Compiles the marshalling extension against this interpreter's and torch's headers.
    None where either lacks them: the C library and the bf16 calls do without."""
    import torch

    out, src = marshal_path(), os.path.join(CSRC, "marshal.cpp")
    if not (force or _stale(out, [src, os.path.join(ROOT, "include", "msa.h")])):
        return out
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    python = sysconfig.get_paths()["include"]
    for header in (os.path.join(python, "Python.h"), os.path.join(inc, "torch", "csrc", "autograd",
                                                                 "python_variable.h")):
        if not os.path.exists(header):
            print("no %s: the 8-bit cache's Python calls are not built" % header, file=sys.stderr)
            return None
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(),
           "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + python,
           src, "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath," + lib]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
