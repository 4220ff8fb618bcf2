"""Builds the in-tree CUDA library libmoe_gb300.so for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel with nvcc, then linked into
_lib/libmoe_gb300.so with a static CUDA runtime so the library loads on a machine without a
GPU (the C ABI can then be inspected; compute calls report a CUDA error). The CPython module of the
8-bit expert calls (csrc/py_experts.c) is built beside it with the host's C compiler; where that or Python's
headers are missing it is left out, with a warning, and those calls raise ImportError.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe_gb300.so")
MODULE_SOURCE = os.path.join(CSRC, "py_experts.c")
MODULE_PATH = os.path.join(HERE, "_experts" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-DMOE_BUILD", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")


def _deps() -> list[str]:
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _stale(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compiles (if needed) and returns the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        if force or _stale(obj, [src] + deps):
            cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stderr}")
            if verbose and res.stderr:
                print(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, sources))
    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
    if force or _stale(MODULE_PATH, [MODULE_SOURCE] + deps):
        _build_module()
    return LIB_PATH


def _build_module() -> None:
    """The CPython module of the 8-bit expert calls, linked to the library beside it."""
    cc, headers = shutil.which("cc") or shutil.which("gcc"), sysconfig.get_paths()["include"]
    if not cc or not os.path.exists(os.path.join(headers, "Python.h")):
        if os.path.exists(MODULE_PATH):
            os.remove(MODULE_PATH)  # it belongs to an earlier library
        warnings.warn(f"built without the 8-bit expert calls: they need a C compiler and {os.path.join(headers, 'Python.h')}")
        return
    tmp = MODULE_PATH + ".tmp"
    cmd = [cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", f"-I{headers}", MODULE_SOURCE, "-o", tmp,
           f"-L{LIB_DIR}", "-lmoe_gb300", "-Wl,-rpath,$ORIGIN/_lib"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"cc failed on {os.path.basename(MODULE_SOURCE)}:\n{res.stderr}")
    os.replace(tmp, MODULE_PATH)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
