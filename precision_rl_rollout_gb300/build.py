"""Build libfp8rl.so in-tree: every csrc/*.cu compiled for sm_103a in parallel
with nvcc, then linked into one shared library beside this file; and beside it the
Python module of the rollout step's calls, _calls.<python>.<torch>.so (csrc/calls.cpp,
host code only, against torch's headers).

    python -m precision_rl_rollout_gb300.build [--force] [--verbose]

No fast-math: the quantizers rely on IEEE division and no flush-to-zero.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libfp8rl.so")
CALLS_STEM = os.path.join(PKG, "_calls")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfp8rl.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def calls_path() -> str:
    """The module of the compiled calls for this Python and this torch: it is compiled
    against both, and one made for others would crash or not load."""
    try:
        import torch
        tag = f"torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    except ImportError:
        tag = "torchless"
    return f"{CALLS_STEM}.{sysconfig.get_config_var('SOABI')}.{tag}.so"


def _newer(target: str, deps) -> bool:
    """target is there and no older than what it is made of."""
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def _calls_up_to_date() -> bool:
    return _newer(calls_path(), [CALLS_SOURCE, os.path.join(INCLUDE, "fp8rl.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _lib_up_to_date() and _calls_up_to_date()


def _build_calls():
    """The compiled calls with the host compiler, against the torch that will import them."""
    import torch
    cxx = shutil.which("g++") or "g++"
    path = calls_path()
    tmp = path + f".tmp{os.getpid()}"
    home = os.path.dirname(os.path.dirname(_nvcc()))
    here = os.path.dirname(torch.__file__)
    inc = [os.path.join(here, "include"), os.path.join(here, "include", "torch", "csrc", "api", "include"),
           os.path.join(home, "include"), sysconfig.get_paths()["include"], INCLUDE]
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *[f"-I{p}" for p in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", CALLS_SOURCE,
           "-o", tmp, "-L" + os.path.join(here, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """-> the library's path.  The library needs no torch: where the compiled calls cannot
    be made it is there all the same, and a warning says why the rollout calls will not be."""
    lib, calls = force or not _lib_up_to_date(), force or not _calls_up_to_date()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        made = ex.submit(_build_calls) if calls else None
        if lib:
            _build_library(verbose, ptxas_verbose)
        try:
            if made:
                made.result()
        except Exception as e:
            if os.path.exists(calls_path()):
                os.remove(calls_path())                # made for another library
            warnings.warn(f"the compiled calls were not built, the rollout step's calls will raise: {e}",
                          RuntimeWarning, stacklevel=2)
    return LIB_PATH


def _build_library(verbose: bool, ptxas_verbose: bool):
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, (r.stdout + r.stderr)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas_verbose))
