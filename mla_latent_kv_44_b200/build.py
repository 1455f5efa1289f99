"""Build libmla.so in-tree with nvcc for sm_100a.

    python -m mla_latent_kv_44_b200.build [--force] [--verbose]

Each csrc/*.cu compiles to an object under _build/ (recompiled when it or a header is newer),
then the objects link into mla_latent_kv_44_b200/libmla.so with the CUDA runtime linked
statically, so the library loads on a machine without a GPU (calls then fail with
MLA_ERR_CUDA) and needs nothing at run time but the NVIDIA driver. A second library,
libmla_testhook.so, differs only in a test define of the attention kernels (one K load of the first
work range is left out in each); only the tests load it. _fast_call.so, through which the Python
binding makes the tree calls, is compiled by g++ against torch's headers; where torch is missing the
libraries are built without it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmla.so")
# Test build: the same library with one K-slab load of the first work range left out
# (MLA_TEST_DROP_ARRIVE), so that the tests can watch a bounded wait run out.
TEST_LIB = os.path.join(PKG, "libmla_testhook.so")
TEST_DEFINE = "-DMLA_TEST_DROP_ARRIVE"
TEST_SOURCES = ("decode_tc.cu", "tree_tc.cu")
FAST_SOURCE = os.path.join(CSRC, "fast_call.cpp")
FAST_LIB = os.path.join(PKG, "_fast_call.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def fast_identity() -> str | None:
    """What the binding's compiled module is built for: this Python and torch (whose C++ interface
    changes with its version). None where one of the things that it needs is missing."""
    spec = importlib.util.find_spec("torch")
    headers = sysconfig.get_paths()["include"]
    if (spec is None or not os.path.exists(os.path.join(headers, "Python.h")) or
            not shutil.which(os.environ.get("CXX", "g++"))):
        return None
    return f"torch {importlib.metadata.version('torch')} {spec.origin}\npython {sys.version}\n"


def fast_command():
    """The g++ command of the binding's compiled module."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    api = os.path.join(root, "include", "torch", "csrc", "api", "include")
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
                os.path.join(root, "include"), api]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
            "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in includes), FAST_SOURCE, "-o", FAST_LIB, f"-L{root}/lib",
            f"-Wl,-rpath,{root}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    jobs = []
    objs = []
    test_objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [src] + headers):
            cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
        if os.path.basename(src) in TEST_SOURCES:
            tobj = os.path.join(BUILD, os.path.basename(src) + ".testhook.o")
            test_objs.append(tobj)
            if force or _stale(tobj, [src] + headers):
                jobs.append([cc, *ARCH, *FLAGS, TEST_DEFINE, "-c", src, "-o", tobj])
        else:
            test_objs.append(obj)

    # built for this torch and Python, as the note beside the objects says
    fast, fast_note = fast_identity(), os.path.join(BUILD, "fast_call.txt")
    fast_job = None
    if fast is None:
        sys.stderr.write("torch, Python's headers or a C++ compiler is missing: the library is built, "
                         "_fast_call.so (the tree calls from Python) is not\n")
    elif force or _stale(FAST_LIB, [FAST_SOURCE] + headers) or _read(fast_note) != fast:
        fast_job = fast_command()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, p

    failed, fast_failed = [], False
    todo = jobs + ([fast_job] if fast_job else [])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as ex:
        for cmd, p in ex.map(run, todo):
            if p.returncode != 0 or ptxas_info or verbose:
                sys.stderr.write(p.stdout + p.stderr)
            if cmd is fast_job:
                fast_failed = p.returncode != 0
            elif p.returncode != 0:
                failed.append(cmd[-3])
    if fast_job and not fast_failed:
        with open(fast_note, "w") as f:
            f.write(fast)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    for lib, parts in ((LIB, objs), (TEST_LIB, test_objs)):
        if force or jobs or _stale(lib, parts):
            cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", lib, *parts]
            if verbose:
                print(" ".join(cmd), flush=True)
            p = subprocess.run(cmd, capture_output=True, text=True)
            if p.returncode != 0:
                raise RuntimeError("link failed:\n" + p.stdout + p.stderr)
    if fast_failed:
        raise RuntimeError(f"{LIB} is built, but {FAST_SOURCE} does not compile")
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills/smem")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    main()
