"""Build libkda.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, linked
with the static CUDA runtime (the library then loads on hosts without a driver); and
_quick.so, the plain calls' way from Python to it (csrc/kda_quick.cpp), beside it where
there are torch, its headers, Python's and g++ to build it with."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
QUICK = os.path.join(HERE, "_quick.so")
QUICK_KEY = os.path.join(HERE, "_quick.key")
QUICK_SOURCE = os.path.join(CSRC, "kda_quick.cpp")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
HEADER = os.path.join(INCLUDE, "kda.h")
UNAVAILABLE = "unavailable: "

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE] + ARCH


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def _lib_up_to_date() -> bool:
    deps = _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [HEADER]
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(deps)


def quick_key() -> str:
    """What _quick.so is built for: the machine, the interpreter and the torch whose headers it saw."""
    import torch
    return "%s %s torch %s abi %d" % (platform.machine(), sys.implementation.cache_tag, torch.__version__,
                                      torch._C._GLIBCXX_USE_CXX11_ABI)


def quick_built_for() -> str:
    """The key of the _quick.so that is there, "unavailable: " and a key where it could not be built, or ""."""
    try:
        with open(QUICK_KEY) as f:
            return f.read()
    except OSError:
        return ""


def _quick_up_to_date() -> bool:
    try:
        key = quick_key()
    except Exception:                      # no torch: nothing to build it against
        return True
    had = quick_built_for()
    if had != UNAVAILABLE + key and (had != key or not os.path.exists(QUICK)):
        return False
    return os.path.getmtime(QUICK_KEY) >= _newest([QUICK_SOURCE, HEADER])


def up_to_date() -> bool:
    return _lib_up_to_date() and _quick_up_to_date()


def _compile_quick():
    """_quick.so against this interpreter's and this torch's headers and libraries."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = QUICK + ".%d.tmp" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + ["-isystem" + d for d in dirs] +
           [QUICK_SOURCE, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (QUICK_SOURCE, " ".join(cmd), r.stderr))
    return tmp


def _build_quick():
    """_quick.so, and what it is for; without it calls take longer, so that a failure is a warning."""
    try:
        key = quick_key()
    except Exception as e:
        warnings.warn("%s is not built: %s" % (QUICK, e), RuntimeWarning)
        return
    try:
        os.replace(_compile_quick(), QUICK)
    except Exception as e:
        warnings.warn("%s is not built: %s" % (QUICK, e), RuntimeWarning)
        key = UNAVAILABLE + key
    with open(QUICK_KEY, "w") as f:
        f.write(key)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    lib, quick = force or not _lib_up_to_date(), force or not _quick_up_to_date()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        done = ex.submit(_build_quick) if quick else None
        if lib:
            _build_lib(ex, verbose, ptxas_info)
        if done:
            done.result()
    return LIB


def _build_lib(ex, verbose, ptxas_info):
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        return obj, r.stderr

    results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for obj, log in results:
            if log.strip():
                print("==", os.path.basename(obj), "\n" + log)
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [cc, "-shared"] + ARCH + ["-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
