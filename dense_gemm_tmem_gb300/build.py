"""Builds the CUDA library in-tree: dense_gemm_tmem_gb300/_build/libdgemm_gb300.so.

Each translation unit is compiled for sm_103a only, in parallel, then linked
with nvcc (static CUDA runtime; the driver is reached at run time through the
runtime's entry-point query, so the library loads on a machine without a GPU).
Beside it, _build/_dgemm_native-*.so: the 8- and 4-bit operators' tensor-facing calls
(csrc/native.cpp) as a Python extension against the installed torch.  Only those
calls need it: where it cannot be built (no host compiler, Python or torch
headers), the library is there all the same and they say why.
"""
from __future__ import annotations

import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libdgemm_gb300.so")
def _torch_version() -> str:
    """torch.__version__, without importing it where its file says it plainly."""
    try:
        where = importlib.util.find_spec("torch").submodule_search_locations[0]
        with open(os.path.join(where, "version.py")) as f:
            return re.search(r"^__version__ = ['\"]([^'\"]+)['\"]", f.read(), re.M).group(1)
    except (AttributeError, OSError):
        return "none"


# the extension links against torch's C++ and Python's C interface: one for each pair
NATIVE = os.path.join(OUT_DIR, "_dgemm_native-%s-torch%s.so"
                      % (sys.implementation.cache_tag, _torch_version()))
NATIVE_SOURCE = os.path.join(CSRC, "native.cpp")
SOURCES = ["api.cu", "simt.cu", "simt_f16.cu", "selftest.cu", "noalloc.cu", "tc2.cu",
           "tc_n256.cu", "tc_n128.cu", "tc_small.cu", "tc_narrow.cu", "tc64.cu",
           "fp8_api.cu", "fp8_quant.cu", "fp8_simt.cu", "fp8_moe.cu", "fp8_tc.cu",
           "fp4_api.cu", "fp4_quant.cu", "fp4_tc.cu", "fp4_row.cu", "ortho.cu", "ortho_tc.cu"]
HEADERS = ["ptx.cuh", "work.cuh", "tc_kernel.cuh", "tc2_kernel.cuh", "tc64_kernel.cuh",
           "tc_launch.cuh", "simt_kernel.cuh", "internal.h", "context.h", "fp8.cuh",
           "fp8_tc_kernel.cuh", "moe_order.h", "fp4.cuh",
           "fp4_quant.cuh", "fp4_tc_kernel.cuh", "ortho.cuh", "ortho_tc_kernel.cuh"]
INCLUDES = ["gemm.h", "gemm_fp8.h", "gemm_fp4.h", "gemm_ortho.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files += [os.path.join(ROOT, "include", h) for h in INCLUDES]
    return files


def _newer(target, files) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def native_up_to_date() -> bool:
    return _newer(NATIVE, _inputs()[-len(INCLUDES):] + [NATIVE_SOURCE])


def build_native() -> str:
    """Compiles the Python extension with the host compiler."""
    os.makedirs(OUT_DIR, exist_ok=True)
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    tmp = NATIVE + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], NATIVE_SOURCE, "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (cmd[0], r.stdout, r.stderr))
    os.replace(tmp, NATIVE)
    return NATIVE


def _native_if_possible():
    try:
        build_native()
    except (OSError, RuntimeError, AttributeError) as e:
        warnings.warn("the 8-bit operators' Python calls are not available: %s" % e)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles and links the library unless it is newer than every source, and the
    extension likewise, whose failure is a warning."""
    native = force or not native_up_to_date()
    if not force and up_to_date():
        if native:
            _native_if_possible()
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        extension = ex.submit(_native_if_possible) if native else None
        objs = list(ex.map(compile_one, SOURCES))
        if extension:
            extension.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
