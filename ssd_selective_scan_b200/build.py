"""Build libssd.so in-tree from csrc/*.cu for sm_100a (B200), and the Python
extension _pycall.so from csrc/pycall.cpp.

    python -m ssd_selective_scan_b200.build [--force] [-v]

Each translation unit is compiled by nvcc into _build/ (in parallel), then
linked into ssd_selective_scan_b200/libssd.so with the static CUDA runtime.
Only sm_100a SASS is generated: the library targets B200 alone.  The extension
is host code against torch's and Python's headers, linked to libssd.so beside
it; it is built anew when either of the two is another version.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

from . import binding

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssd.so")
PYCALL_SRC = os.path.join(CSRC, "pycall.cpp")
PYCALL = os.path.join(PKG, "_pycall.so")
PYCALL_STAMP = os.path.join(BUILD, "pycall.built_for")   # what the built one is for
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def _fresh(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _fresh(LIB, _deps())


def _pycall_fresh() -> bool:
    if not _fresh(PYCALL, [PYCALL_SRC, os.path.join(INCLUDE, "ssd.h"), os.path.join(INCLUDE, "ssd_diag.h"), os.path.abspath(__file__)]):
        return False
    try:
        with open(PYCALL_STAMP) as f:
            return f.read() == binding.pycall_target()
    except OSError:
        return False


def _build_pycall(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    target = binding.pycall_target()
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = PYCALL + f".tmp{os.getpid()}"
    cmd = [CXX, "-O2", "-std=c++17", f'-DSSD_BUILT_FOR="{target}"', "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include"), PYCALL_SRC, "-o", tmp,
           "-L", PKG, "-l:" + os.path.basename(LIB), "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on {PYCALL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYCALL)
    with open(PYCALL_STAMP, "w") as f:
        f.write(target)


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if force or not up_to_date():
        _build_lib(verbose, ptxas_info)
    if force or not _pycall_fresh():
        _build_pycall(verbose)
    return LIB


def _build_lib(verbose: bool, ptxas_info: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose or ptxas_info, extra), _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args(argv)
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    sys.exit(main())
