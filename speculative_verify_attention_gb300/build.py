"""Build libkvq8attn.so in-tree with nvcc for sm_103a (GB300).

Every .cu file under csrc/ is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo`` and linked into one shared
library next to this file.  csrc/calls.cpp, the binding's argument checks of the calls that stand in steps
of a few microseconds, is compiled beside them with the host compiler against torch's headers, and linked
to that library.  No CMake, no torch extension machinery.  The C library is linked first and needs neither
torch nor Python; where torch is not installed it is all that is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libkvq8attn.so")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
CALLS_PATH = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [CALLS_SOURCE, os.path.join(INCLUDE, "kvq8attn.h")]


def _torch_dir():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def needs_build() -> bool:
    paths = [LIB_PATH] + ([CALLS_PATH] if _torch_dir() else [])
    if not all(os.path.exists(p) for p in paths):
        return True
    t = min(os.path.getmtime(p) for p in paths)
    return any(os.path.getmtime(p) > t for p in _deps())


def _link(path: str, compiler: list, rest: list) -> None:
    tmp = path + f".{os.getpid()}.tmp"
    r = subprocess.run([*compiler, "-shared", "-o", tmp, *rest], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link the library; returns its path."""
    if not force and not needs_build():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    calls_obj = os.path.join(BUILD_DIR, "calls.cpp.o")
    torch_dir = _torch_dir()

    def compile_calls():
        include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], INCLUDE]
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *[f"-I{d}" for d in include], "-c", CALLS_SOURCE, "-o", calls_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the host compiler failed for {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")

    with cf.ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        calls = ex.submit(compile_calls) if torch_dir else None
        objs = list(ex.map(compile_one, srcs))
        # the C library first: it needs nothing of torch or Python
        _link(LIB_PATH, [nvcc, *ARCH], [*objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"])
        if calls:
            calls.result()
    if torch_dir:
        _link(CALLS_PATH, [os.environ.get("CXX", "g++")], [calls_obj, f"-L{HERE}", "-lkvq8attn", f"-L{os.path.join(torch_dir, 'lib')}",
                                                            "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"])
    else:
        sys.stderr.write("torch is not installed: the C library alone was built\n")
    return LIB_PATH


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=True, verbose=v or bool(extra), extra_flags=extra))
