"""Build ``libkda.so`` in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in its own nvcc process (in parallel), then one
link step produces the shared library next to this file.  The CUDA runtime is
linked statically, so the library needs only the NVIDIA driver at run time.
Beside it the host compiler builds ``_paged_fast.so``, the short way from Python
into the paged calls; the library does not need it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
FAST_SRC = os.path.join(HERE, "csrc_py", "paged_fast.cpp")
FAST = os.path.join(HERE, "_paged_fast.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA library needs the CUDA 13 toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_fast(force: bool = False) -> str:
    """Compile csrc_py/paged_fast.cpp against the installed torch; returns the module's path."""
    import torch
    from torch.utils import cpp_extension

    stamp = os.path.join(BUILD, "torch_version")
    version = torch.__version__ + " " + sysconfig.get_python_version()
    built_for = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and built_for == version and not _stale(FAST, [FAST_SRC, __file__] + _headers()):
        return FAST
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], cuda] + cpp_extension.include_paths()
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = FAST + f".tmp{os.getpid()}"
    cmd = (["g++", "-std=c++17", "-O2", "-fPIC", "-shared", FAST_SRC, "-o", tmp] + [f"-I{d}" for d in dirs] +
           [f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FAST)
    with open(stamp, "w") as f:
        f.write(version)
    return FAST


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile every csrc/*.cu and link libkda.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    flags = NVCC_FLAGS + list(extra_flags or [])
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs + [__file__]):
            jobs.append([nvcc()] + ARCH + flags + ["-c", s, "-o", o])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = [ex.submit(subprocess.run, j, capture_output=True, text=True) for j in jobs]
            for j, f in zip(jobs, futs):
                r = f.result()
                if verbose and (r.stdout or r.stderr):
                    print(r.stdout, r.stderr)
                if r.returncode != 0:
                    raise RuntimeError(f"nvcc failed: {' '.join(j)}\n{r.stdout}\n{r.stderr}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_fast(force=True))
