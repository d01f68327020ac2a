"""Builds ``libswiglu_mlp.so`` in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel to ``_build/*.o`` and the objects
are linked into one shared library (CUDA runtime linked statically).  Objects
are rebuilt only when a source or header is newer than them.  The CPython module
``_binding`` (plain C, gcc) is linked against that library beside it, after it:
the library's C users need no Python headers.  It keeps to the stable ABI of
CPython 3.10, so that any later interpreter may load it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libswiglu_mlp.so")
BINDING = os.path.join(HERE, "_binding.abi3.so")
SOURCES = ["api.cu", "api_experts.cu", "k_grouped.cu", "k_grouped_mx4.cu", "k_wgrad.cu", "k_mx4.cu", "k_reduce.cu", "k_store.cu", "k_swiglu.cu", "k_splitk.cu", "k_fp8.cu", "k_gemv.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = _headers()
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({' '.join(cmd)}):\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, flush=True)

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    src = os.path.join(CSRC, "binding.c")
    if force or _stale(BINDING, [src] + hdrs):
        tmp = BINDING + f".tmp{os.getpid()}"
        run(["gcc", "-O2", "-shared", "-fPIC", "-Wall", "-DPy_LIMITED_API=0x030A0000", "-I", INCLUDE,
             "-I", sysconfig.get_paths()["include"], src, "-o", tmp,
             "-L", HERE, "-lswiglu_mlp", "-Wl,-rpath,$ORIGIN"])
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
