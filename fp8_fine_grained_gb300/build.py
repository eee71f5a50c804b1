"""Build libfp8fg.so (the C-ABI library) in-tree with nvcc for sm_103a, and the
binding's CPython helper _tensors.so with the host compiler.

Each translation unit compiles in parallel; the CUDA objects link into one
shared library with the CUDA runtime linked statically, so the library loads
on a machine without a GPU driver (nothing runs until a call is made). The
helper reads the metadata of torch tensors and is compiled against the
installed torch; it is made anew for another torch or Python. Only the operators
between a gated MLP's GEMMs need it, so where it cannot be made (no headers)
build() says so and leaves the library.
"""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfp8fg.so")
HELPER = os.path.join(HERE, "_tensors.so")
HELPER_SOURCE = os.path.join(CSRC, "tensors.cpp")
SOURCES = ["capi.cu", "quant.cu", "gemm.cu", "gemm_mx.cu", "moe.cu", "norm.cu", "gemm_gated.cu", "gated_bwd.cu",
           "clip.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files.append(os.path.join(INCLUDE, "fp8fg.h"))
    return max(os.path.getmtime(f) for f in files)


def helper_command(out):
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    torch = spec.submodule_search_locations[0]
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
            sysconfig.get_paths()["include"], HELPER_SOURCE, "-o", out, "-L", lib, "-Wl,-rpath," + lib,
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]


def _made_for():
    """What the helper depends on beside its sources: the compiler's command,
    Python's ABI and torch's version (read from its file: importing it is slow)."""
    command = helper_command("")
    version = os.path.join(importlib.util.find_spec("torch").submodule_search_locations[0], "version.py")
    with open(version) as f:
        return "\n".join(command + [str(sysconfig.get_config_var("SOABI")), f.read()])


def build_helper(force=False):
    made_for, stamp = _made_for(), os.path.join(BUILD, "tensors.made_for")
    newest = max(os.path.getmtime(f) for f in (HELPER_SOURCE, os.path.join(INCLUDE, "fp8fg.h")))
    if not force and os.path.exists(HELPER) and os.path.getmtime(HELPER) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == made_for:
                return HELPER
    tmp = HELPER + ".tmp.%d" % os.getpid()
    try:
        r = subprocess.run(helper_command(tmp), capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError("%s: no host compiler (%s)" % (HELPER_SOURCE, e))
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (HELPER_SOURCE, r.stdout, r.stderr))
    # (the record goes first and comes back last: a build cut short in between is made again)
    if os.path.exists(stamp):
        os.remove(stamp)
    os.replace(tmp, HELPER)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(made_for)
    return HELPER


def build(force=False, verbose=False, extra=(), strict=False):
    """The library, and the helper beside it. A helper that cannot be made is a
    warning (an error with `strict`)."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        helper = ex.submit(build_helper, force)
        lib = build_lib(force, verbose, extra)
        try:
            helper.result()
        except RuntimeError as e:
            if strict:
                raise
            warnings.warn("the operators between a gated MLP's GEMMs are not available: %s" % e, RuntimeWarning)
    return lib


def build_lib(force=False, verbose=False, extra=()):
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stdout.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
