"""Builds libsv.so in-tree with nvcc for sm_103a (GB300), and the Python
extension over it.

Each .cu file under csrc/ is compiled in parallel to an object, then linked
into one shared library with the CUDA runtime linked statically, so the
library only needs the driver at run time.  csrc/py_calls.cpp is compiled
beside them against the installed torch.  Output: csrc/_build/libsv.so and
csrc/_build/sv_calls.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
# SV_DEBUG=1 builds the self-checking variant (-DSV_DEBUG) into its own folder.
DEBUG = os.environ.get("SV_DEBUG", "") == "1"
OUT_DIR = os.path.join(CSRC, "_build_debug" if DEBUG else "_build")
LIB = os.path.join(OUT_DIR, "libsv.so")
CALLS = os.path.join(OUT_DIR, "sv_calls.so")
CALLS_FOR = os.path.join(OUT_DIR, "sv_calls.for")   # what it was built against
CALLS_SRC = os.path.join(CSRC, "py_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "sv.h"))
    return hs


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def calls_target() -> str:
    """The interpreter and the torch that the extension has to match."""
    import torch
    return f"Python {sys.version.split()[0]}, torch {torch.__version__}"


def calls_built_for() -> str:
    try:
        with open(CALLS_FOR) as f:
            return f.read()
    except OSError:
        return "an unknown Python and torch"


def _calls_compile(obj):
    import torch   # the headers and the ABI that the extension has to match
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    inc = [root, os.path.join(root, "torch", "csrc", "api", "include"), cuda, sysconfig.get_paths()["include"], INCLUDE]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + \
        [x for d in inc for x in ("-isystem" if d != INCLUDE else "-I", d)] + ["-c", CALLS_SRC, "-o", obj]


def _calls_link(obj, out):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L", OUT_DIR, "-lsv", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN:" + lib]


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    flags = NVCC_FLAGS + (["-DSV_DEBUG"] if DEBUG else []) + list(extra_flags or [])
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([nvcc] + ARCH + flags + ["-c", src, "-o", obj])

    calls_obj = os.path.join(OUT_DIR, "py_calls.o")
    calls = force or calls_built_for() != calls_target() or _stale(calls_obj, [CALLS_SRC, os.path.join(INCLUDE, "sv.h")])
    if calls:
        jobs.insert(0, _calls_compile(calls_obj))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compilation failed: " + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-ldl", "-lpthread", "-lrt"])
        os.replace(tmp, LIB)
    if calls or _stale(CALLS, [calls_obj]):
        run(_calls_link(calls_obj, CALLS + ".tmp"))
        os.replace(CALLS + ".tmp", CALLS)
        with open(CALLS_FOR, "w") as f:
            f.write(calls_target())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
