"""Builds libdfl2.so in-tree from csrc/*.cu for sm_103a with nvcc, and the Python
extension _calls.so from csrc/calls.cpp with the host compiler.

Each translation unit is compiled in parallel, then linked into one shared
library that exports the C ABI of include/dfl2.h; the extension is linked
against it and torch.  The library needs no torch: without it it is all that is
built, and where the extension cannot be built the library is there all the same.
Each is rebuilt only when a source or header of its own is newer, the extension
for another Python or torch too.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdfl2.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_lock = threading.Lock()


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the dfl2 CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(out, deps) -> bool:
    """Whether `out` is there and no older than what it is made from."""
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(p) <= t
               for p in [*deps, *glob.glob(os.path.join(INCLUDE, "*.h")), os.path.abspath(__file__)])


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def lib_fresh() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def calls_made_with() -> str:
    """What the extension's binary interface depends on besides its sources."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # one that was not installed as a package
        import torch
        version = torch.__version__
    return f"{sysconfig.get_config_var('SOABI')}, torch {version}\n"


def _calls_note():
    return os.path.join(BUILD, "calls.txt")


def calls_fresh() -> bool:
    if not (_newer(CALLS, [CALLS_SRC]) and os.path.exists(_calls_note())):
        return False
    with open(_calls_note()) as f:
        return f.read() == calls_made_with()


def is_fresh() -> bool:
    return lib_fresh() and (calls_fresh() or not has_torch())


def cflags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr", *extra]


def calls_cmds(cc: str, obj: str, out: str):
    """The commands that compile and link _calls.so."""
    import torch
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("g++ not found: the Python extension of dfl2 cannot be built")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda,
            sysconfig.get_paths()["include"]]
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *(x for d in dirs for x in ("-isystem" if d != INCLUDE else "-I", d)),
             "-c", CALLS_SRC, "-o", obj],
            [cxx, "-shared", "-o", out, obj, "-L", PKG, "-ldfl2", "-Wl,-rpath,$ORIGIN",
             "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile and link libdfl2.so and, with torch, _calls.so; returns the first one's path."""
    with _lock:
        lib = force or not lib_fresh()
        calls = has_torch() and (force or not calls_fresh())
        if not (lib or calls):
            return LIB
        os.makedirs(BUILD, exist_ok=True)
        cc = nvcc()

        def compile_one(src, cmd):
            if verbose:
                print(" ".join(cmd))
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed on "
                                   f"{os.path.basename(src)}:\n{r.stderr}")
            if verbose and r.stderr:
                print(r.stderr)

        def compile_cu(src):
            obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
            compile_one(src, [cc, *cflags(extra), "-c", src, "-o", obj])
            return obj

        calls_tmp = CALLS + f".tmp{os.getpid()}"

        def compile_calls():
            compile_cmd, link_cmd = calls_cmds(cc, os.path.join(BUILD, "calls.o"), calls_tmp)
            compile_one(CALLS_SRC, compile_cmd)
            return link_cmd

        def link(cmd, tmp, out):
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, out)

        with cf.ThreadPoolExecutor(max_workers=8) as ex:
            calls_link = ex.submit(compile_calls) if calls else None
            if lib:
                objs = list(ex.map(compile_cu, _sources()))
                tmp = LIB + f".tmp{os.getpid()}"
                link([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl",
                      "-lpthread"], tmp, LIB)
            if calls:
                link(calls_link.result(), calls_tmp, CALLS)
                with open(_calls_note(), "w") as f:
                    f.write(calls_made_with())
        return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else ()))
