"""In-tree build of ``libnt.so`` for sm_103a with nvcc, and of the compiled
part of its Python binding (``_nt_binding``, host code only) with g++.

Each ``csrc/*.cu`` translation unit compiles in parallel to an object under
``_build/``; the objects link into ``libnt.so`` beside this file with the
CUDA runtime linked statically, so the library loads on a machine without a
GPU driver (only the C-ABI symbols are needed there).  The library needs nvcc
and its host compiler only: without torch, whose headers the binding takes, it
is built alone.  A stamp of the source hashes and the host architecture for
each of the two (the binding's with the versions of Python and torch) skips
rebuilds that would change nothing.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnt.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_nt_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
STAMP = os.path.join(BUILD, "stamp.txt")
BINDING_STAMP = os.path.join(BUILD, "binding_stamp.txt")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH_FLAGS + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                       "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"),
                 os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"),
                 shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set CUDA_HOME or NVCC")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _torch():
    """The torch module, None without one."""
    try:
        import torch
        return torch
    except ImportError:
        return None


def _digest(about, files) -> str:
    h = hashlib.sha256()
    h.update(platform.machine().encode())
    h.update(" ".join(about).encode())
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _current(out: str, stamp: str, digest: str) -> bool:
    if not os.path.exists(out) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read().strip() == digest


def _stamp(stamp: str, digest: str) -> None:
    with open(stamp, "w") as f:
        f.write(digest)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + CFLAGS + list(extra) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding(torch) -> None:
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH_FLAGS + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libnt.so and, where there is torch, the binding;
    returns the library's path.  A binding that fails to compile is reported
    when the library stands."""
    os.makedirs(BUILD, exist_ok=True)
    srcs, header = sources(), os.path.join(INCLUDE, "nt.h")
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))) + [header]
    digest = _digest(CFLAGS, srcs + headers)
    library = force or not _current(LIB, STAMP, digest)
    torch = _torch()
    if torch is not None:
        b_digest = _digest([sys.version, torch.__version__], [BINDING_SRC, header])
    binding = torch is not None and (force or not _current(BINDING, BINDING_STAMP, b_digest))
    jobs = min(len(srcs) + 1, max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bound = ex.submit(_compile_binding, torch) if binding else None
        if library:
            _link(list(ex.map(lambda s: _compile(s, extra_flags), srcs)))
            _stamp(STAMP, digest)
        if bound is not None:
            bound.result()
            _stamp(BINDING_STAMP, b_digest)
    if verbose and (library or binding):
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
