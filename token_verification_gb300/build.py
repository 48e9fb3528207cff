"""Build libspecverify.so (the C-ABI CUDA library) and _binding.so (the Python
binding's short way into it, against the installed PyTorch) in-tree.  The
library needs nvcc alone; without PyTorch there is no binding to build.

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
BUILT_FOR = os.path.join(BUILD, "binding.txt")  # the Python and PyTorch that _binding.so was built for
SOURCES = ["api.cu", "sv_verify.cu", "sv_finalize.cu", "sv_filter.cu", "sv_tree.cu", "sv_noalloc.cu", "sv_ngram.cu",
           "sv_top.cu", "sv_toprows.cu", "sv_distill.cu", "sv_reorder.cu",
           "sv_cache.cu", "sv_attend.cu", "sv_attend_many.cu", "sv_attend_rows.cu"]
HEADERS = ["sv_common.cuh", "sv_launch.h", "sv_rows.cuh", "sv_stream.cuh", "sv_vec.cuh", "sv_select.cuh",
           "sv_cache.cuh", "sv_attend.cuh", "sv_attend_tc.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I" + os.path.join(ROOT, "include")]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def _newer(target, sources):
    """Whether target is there and no older than its sources, the header and this file."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    files = [os.path.join(CSRC, s) for s in sources]
    files += [os.path.join(ROOT, "include", "spec_verify.h"), os.path.abspath(__file__)]
    return all(os.path.getmtime(f) <= t for f in files)


def lib_up_to_date():
    return _newer(LIB, SOURCES + HEADERS)


def torch_dir():
    """The installed PyTorch's folder (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _binding_for(torch_dir):
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "%s\n%s\n%s" % (sysconfig.get_config_var("SOABI"), torch_dir, f.read())


def binding_up_to_date():
    """Whether _binding.so is current, for the Python and PyTorch that are installed now."""
    at = torch_dir()
    if at is None:
        return True
    if not (_newer(BINDING, ["binding.cpp"]) and os.path.exists(BUILT_FOR)):
        return False
    with open(BUILT_FOR) as f:
        return f.read() == _binding_for(at)


def up_to_date():
    return lib_up_to_date() and binding_up_to_date()


def build_binding(cc: str, torch_dir: str) -> str:
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
    with open(BUILT_FOR, "w") as f:
        f.write(_binding_for(torch_dir))
    return BINDING


def build_lib(cc: str, verbose: bool = False, ptxas_info: bool = False) -> str:
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

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Bring both up to date. A binding that fails to build is an error, but not one that keeps
    the library from being built."""
    with_lib, at = force or not lib_up_to_date(), torch_dir()
    with_binding = at is not None and (force or not binding_up_to_date())
    if not (with_lib or with_binding):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    with ThreadPoolExecutor(1) as ex:
        binding = ex.submit(build_binding, cc, at) if with_binding else None
        if with_lib:
            build_lib(cc, verbose, ptxas_info)
        if binding is not None:
            binding.result()
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
