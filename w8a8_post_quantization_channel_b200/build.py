"""Builds libsq.so in-tree from csrc/*.cu with nvcc for sm_100a, and the
binding's native part, _binding.so, from csrc/sq_binding.cpp.

Usage: python -m w8a8_post_quantization_channel_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import glob
import hashlib
import mmap
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsq.so")
BINDING_SRC = os.path.join(CSRC, "sq_binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
# No fast-math: IEEE division/sqrt and no FMA contraction keep every
# rounding step identical to the method's fp32 definition.
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC,-O2",
           "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = [os.environ.get("NVCC", ""), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc") or ""]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources() -> list[str]:
    """What libsq.so is made from."""
    files = glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h"))
    return sorted(files + glob.glob(os.path.join(INCLUDE, "*.h")))


def _key(files: list[str], *more: str) -> str:
    """A text of the files' contents and of `more`, which a binary carries: one
    made from anything else is not taken for up to date, whatever its time."""
    h = hashlib.sha256()
    for part in (*(os.path.basename(f) for f in files), *more):
        h.update(part.encode() + b"\0")
    for f in files:
        with open(f, "rb") as src:
            h.update(hashlib.sha256(src.read()).digest())
    return "sq-built-from:" + h.hexdigest()


def _carries(path: str, key: str) -> bool:
    try:
        with open(path, "rb") as f, mmap.mmap(f.fileno(), 0, access=mmap.ACCESS_READ) as m:
            return m.find(key.encode()) >= 0
    except (OSError, ValueError):  # missing, or empty
        return False


@contextlib.contextmanager
def _alone():
    """One build of this tree at a time, over threads and processes."""
    os.makedirs(OBJ, exist_ok=True)
    with open(os.path.join(OBJ, "lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _binding_key() -> str:
    import sysconfig

    import torch
    return _key([BINDING_SRC, os.path.join(INCLUDE, "sq.h")], torch.__version__, str(torch.version.git_version),
                str(torch.compiled_with_cxx11_abi()), str(sysconfig.get_config_var("SOABI")))


def build_binding(force: bool = False) -> str:
    """Compile _binding.so against the torch that runs this."""
    if not force and not os.path.exists(BINDING_SRC) and os.path.exists(BINDING):
        return BINDING  # a tree without sources
    if not force and _carries(BINDING, _binding_key()):
        return BINDING
    with _alone():
        key = _binding_key()
        if not force and _carries(BINDING, key):  # made by another one meanwhile
            return BINDING
        import sysconfig

        import torch
        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(nvcc()))
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DSQ_BUILD_KEY="{key}"',
               "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
               "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp, "-L", os.path.join(root, "lib"),
               "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ldl"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)
        return BINDING


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every csrc/*.cu and link libsq.so (static cudart)."""
    if not force and not _sources() and os.path.exists(LIB):
        return LIB  # a tree without sources
    flags = " ".join([*ARCH, *(f for f in NVFLAGS if f not in (INCLUDE, CSRC))])
    if not force and _carries(LIB, _key(_sources(), flags)):
        return LIB
    with _alone():
        key = _key(_sources(), flags)
        if not force and _carries(LIB, key):  # made by another one meanwhile
            return LIB
        srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
        extra = [f'-DSQ_BUILD_KEY="{key}"'] + (["-Xptxas", "-v"] if verbose_ptxas else [])
        with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
            objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
    print(build_binding(force="--force" in sys.argv))
