"""Build libspecverify.so (the C-ABI CUDA library) and _binding.so (the Python
binding's short way into it, against the installed PyTorch) in-tree.

Every translation unit is compiled for sm_103a only, in parallel, then linked
against the shared CUDA runtime (the same libcudart.so.13 that PyTorch loads).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecverify.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "sv_verify.cu", "sv_finalize.cu", "sv_filter.cu", "sv_tree.cu", "sv_noalloc.cu", "sv_ngram.cu",
           "sv_top.cu", "sv_toprows.cu", "sv_distill.cu", "sv_reorder.cu"]
HEADERS = ["sv_common.cuh", "sv_launch.h", "sv_rows.cuh", "sv_stream.cuh", "sv_vec.cuh", "sv_select.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I" + os.path.join(ROOT, "include")]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(CSRC, "binding.cpp"))
    files.append(os.path.join(ROOT, "include", "spec_verify.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date():
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_binding(cc: str) -> str:
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    torch_inc = os.path.join(torch_dir, "include")
    torch_lib = os.path.join(torch_dir, "lib")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    tmp = BINDING + ".%d.tmp" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I" + torch_inc, "-I" + os.path.join(torch_inc, "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + cuda_inc,
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L" + torch_lib,
           "-Wl,-rpath," + torch_lib, "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for binding.cpp:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, cc)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
