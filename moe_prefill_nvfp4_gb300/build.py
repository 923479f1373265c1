"""Build the in-tree CUDA library ``lib/libmoe_prefill.so`` for sm_103a with nvcc.

Each ``csrc/*.cu`` file is compiled in parallel (``-gencode arch=compute_103a,code=sm_103a``),
then linked into one shared library against the shared CUDA runtime (the same libcudart that
PyTorch loads, so streams and the primary context are shared) and nothing else: every product,
the shared expert's dense ones included, runs in this library's own kernels.  No cmake, no torch
extension machinery: the library exports a plain C ABI (``include/moe_prefill.h``).
``csrc/fp8_call.c``, the FP8 calls' argument marshalling, becomes the extension module
``lib/_fp8_call<suffix>.so`` beside it, one for each interpreter that built it (the host compiler
and Python's own headers, no others).  Where it cannot be built the library still is:
``build`` warns, and the FP8 calls, which need it, fail with the compiler's message.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIBNAME = "libmoe_prefill.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def lib_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def call_path() -> str:
    return os.path.join(LIBDIR, "_fp8_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


CALL_SOURCE = os.path.join(CSRC, "fp8_call.c")
HEADER = os.path.join(ROOT, "include", "moe_prefill.h")


def _newer(path: str, inputs) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(f) for f in inputs)


def _library_up_to_date() -> bool:
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return _newer(lib_path(), sources() + headers + [HEADER, os.path.abspath(__file__)])


def _call_up_to_date() -> bool:
    return _newer(call_path(), [CALL_SOURCE, HEADER, os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _library_up_to_date() and _call_up_to_date()


def build_call_module() -> str:
    """Compiles the FP8 calls' argument marshalling for this interpreter; raises with the compiler's message."""
    tmp = call_path() + ".tmp"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I",
           os.path.join(ROOT, "include"), CALL_SOURCE, "-o", tmp, "-L", LIBDIR, "-l:" + LIBNAME, "-Wl,-rpath,$ORIGIN"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stderr if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is not None:
        if os.path.exists(call_path()):  # (of older sources)
            os.remove(call_path())
        raise RuntimeError(f"building the FP8 calls' module failed:\n{failed}")
    os.replace(tmp, call_path())
    return call_path()


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link; returns the library path.  Rebuilds only what has a newer source."""
    if force or not _library_up_to_date():
        _build_library(verbose, ptxas_verbose)
    if force or not _call_up_to_date():
        try:
            build_call_module()
        except RuntimeError as e:
            warnings.warn(f"no FP8 calls: {e}", RuntimeWarning)
    return lib_path()


def _build_library(verbose: bool, ptxas_verbose: bool) -> None:
    nvcc = nvcc_path()
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = lib_path() + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results] + [
        "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib_path())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
