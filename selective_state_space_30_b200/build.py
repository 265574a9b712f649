"""Build the CUDA library libssmscan.so in-tree for sm_100a.

    python -m selective_state_space_30_b200.build [--force] [--debug]

The library is the product: kernels plus the C ABI declared in
include/ssm_scan.h.  Each translation unit compiles in parallel, and beside them
_front.so, the compiled torch front ends of the slot and convolution operators
(csrc/front.cpp), which call the library's entry points.  Without torch the
library is built alone.  --debug builds
libssmscan_debug.so from the same sources with SSM_DEBUG defined: the scan
kernels then check their indices against the buffers they touch and record
SSM_ERR_BOUNDS in the device status word instead of making a bad access.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libssmscan.so")
LIB_DEBUG = os.path.join(HERE, "libssmscan_debug.so")
FRONT = os.path.join(HERE, "_front.so")
BUILD_DIR = os.path.join(HERE, "_build")
FRONT_STAMP = os.path.join(BUILD_DIR, "_front.txt")
BUILD_DIR_DEBUG = os.path.join(HERE, "_build_debug")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v", f"-I{INCLUDE}"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src: str, extra, build_dir=BUILD_DIR) -> str:
    obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
    log = obj + ".ptxas.txt"
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr[-4000:]}")
    return obj


def _front_wants():
    """What _front.so is built for beside its sources, torch's version and Python's; None without torch."""
    try:
        return f"torch {importlib.metadata.version('torch')}, Python {sys.version_info.major}.{sys.version_info.minor}"
    except importlib.metadata.PackageNotFoundError:
        return None


def _front_stale() -> bool:
    """Whether the front ends are to be built: sources newer than they are, or another torch or Python."""
    wants = _front_wants()
    if wants is None:
        return False
    try:
        with open(FRONT_STAMP) as f:
            built = f.read()
    except OSError:
        built = None
    return built != wants or _stale(FRONT, [os.path.join(CSRC, "front.cpp"), os.path.join(INCLUDE, "ssm_scan.h")])


def _compile_front() -> str:
    """The compiled front ends: host C++ against torch's headers; torch's libraries are loaded before it."""
    import sysconfig
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = FRONT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{INCLUDE}",
           *(f"-I{p}" for p in include_paths("cuda")), f"-I{sysconfig.get_paths()['include']}",
           os.path.join(CSRC, "front.cpp"), "-o", tmp, *(f"-L{p}" for p in library_paths("cuda")),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on front.cpp:\n{res.stderr[-4000:]}")
    os.replace(tmp, FRONT)
    os.makedirs(os.path.dirname(FRONT_STAMP), exist_ok=True)
    with open(FRONT_STAMP, "w") as f:
        f.write(_front_wants() or "")
    return FRONT


def _stale(lib, outputs_newer_than):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in outputs_newer_than)


def build(force: bool = False, extra=(), debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    build_dir = BUILD_DIR_DEBUG if debug else BUILD_DIR
    extra = list(extra) + (["-DSSM_DEBUG"] if debug else [])
    deps = sources() + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + \
        [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    if force or _stale(lib, deps):
        os.makedirs(build_dir, exist_ok=True)
        srcs = sources()
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
            objs = list(ex.map(lambda s: _compile(s, extra, build_dir), srcs))
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr[-4000:]}")
        os.replace(tmp, lib)
    # the library stands by itself: the front ends come behind it, and only where torch is
    if _front_stale() or (force and _front_wants() is not None):
        _compile_front()
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, debug="--debug" in sys.argv))
