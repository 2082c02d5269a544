"""Builds libmladecode.so in-tree for sm_103a (no cmake; parallel nvcc), and the
CPython module _mla_calls.so that passes torch tensors to it.  The library needs
nvcc and a C++ compiler; the module is left out where there is no CUDA build of
torch with its headers, or no Python.h.

    python -m paged_mla_decode_08_gb300.build      # or build() from Python

Objects go to ``_build/`` at the repository root, the library to
``paged_mla_decode_08_gb300/lib/``.  Source-hash stamps skip the build of
what did not change.
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmladecode.so")
CALLS = os.path.join(LIBDIR, "_mla_calls.so")

CUDA_SOURCES = ["mla_abi.cu", "mla_sm103.cu", "mla_combine.cu", "mla_noalloc.cu", "mla_block_table.cu",
                "mla_plan_device.cu", "mla_kv_write.cu", "mla_norm_quant.cu", "mla_gemm_fp8.cu",
                "mla_prefill.cu", "mla_prompt_rows.cu"]
CXX_SOURCES = ["mla_plan.cpp"]
CALLS_SOURCE = "mla_torch_calls.cpp"  # built against this machine's Python and torch
HEADERS = ["mla_internal.h", "mla_prompt.h", "per_device.h", "sm103_ptx.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", INCLUDE]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str | None:
    """The folder of a CUDA torch with its headers, without importing it; None:
    there is none, or no Python.h, so the module cannot be built."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    path = os.path.dirname(spec.origin)
    needed = [os.path.join(path, "include", "c10", "cuda", "CUDAStream.h"), os.path.join(path, "lib", "libc10_cuda.so"),
              os.path.join(path, "lib", "libtorch_python.so"), os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return path if all(os.path.exists(f) for f in needed) else None


def _stamp(sources, extra: str) -> str:
    h = hashlib.sha256()
    for f in sorted(sources):
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    with open(os.path.join(INCLUDE, "mla_decode.h"), "rb") as fh:
        h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + CXX_FLAGS).encode())
    h.update((os.uname().machine + extra).encode())
    return h.hexdigest()


def _fresh(product: str, stamp_file: str, stamp: str) -> bool:
    if not os.path.exists(product) or not os.path.exists(stamp_file):
        return False
    with open(stamp_file) as fh:
        return fh.read().strip() == stamp


def _finish(tmp: str, product: str, stamp_file: str, stamp: str) -> None:
    os.replace(tmp, product)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)


def _run(cmd, log):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if log is not None:
        log.append((cmd, r.stdout))
    if r.returncode != 0:
        raise RuntimeError(f"build step failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}")
    return r.stdout


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA/C++ source and link the shared library (returns its
    path), and the torch module where it can be built."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    torch_dir = _torch_dir()
    lib_stamp, lib_stamp_file = _stamp(CUDA_SOURCES + CXX_SOURCES + HEADERS, ""), os.path.join(BUILD, "stamp")
    lib_stale = force or not _fresh(LIB, lib_stamp_file, lib_stamp)
    calls_stamp_file, calls_stale = os.path.join(BUILD, "stamp_calls"), False
    if torch_dir is None:
        if os.path.exists(CALLS):  # of a torch that is gone
            os.remove(CALLS)
    else:
        calls_stamp = _stamp([CALLS_SOURCE], sys.version + importlib.metadata.version("torch") + torch_dir)
        calls_stale = force or not _fresh(CALLS, calls_stamp_file, calls_stamp)
    if not lib_stale and not calls_stale:
        return LIB
    nvcc, cxx = _nvcc(), os.environ.get("CXX", "g++")
    log: list = []
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        jobs, objs, calls_job = [], [], None
        if lib_stale:
            for src in CUDA_SOURCES + CXX_SOURCES:
                obj = os.path.join(BUILD, src + ".o")
                objs.append(obj)
                compiler = [nvcc, *ARCH, *NVCC_FLAGS] if src in CUDA_SOURCES else [cxx, *CXX_FLAGS]
                jobs.append(ex.submit(_run, [*compiler, "-c", os.path.join(CSRC, src), "-o", obj], log))
        if calls_stale:
            calls_obj = os.path.join(BUILD, CALLS_SOURCE + ".o")
            cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
            include = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                       os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
            calls_job = ex.submit(_run, [cxx, *CXX_FLAGS, *(a for d in include for a in ("-isystem", d)), "-c",
                                         os.path.join(CSRC, CALLS_SOURCE), "-o", calls_obj], log)
        for job in jobs:
            job.result()
        if lib_stale:
            tmp = LIB + ".tmp"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], log)
            _finish(tmp, LIB, lib_stamp_file, lib_stamp)
        if calls_job:
            calls_job.result()
            tmp = CALLS + ".tmp"
            _run([cxx, "-shared", "-o", tmp, calls_obj, "-L" + LIBDIR, "-l:libmladecode.so", "-Wl,-rpath,$ORIGIN",
                  "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], log)
            _finish(tmp, CALLS, calls_stamp_file, calls_stamp)
    with open(os.path.join(BUILD, "build.log"), "w") as fh:
        for cmd, out in log:
            fh.write("$ " + " ".join(cmd) + "\n" + out + "\n")
    if verbose:
        for cmd, out in log:
            print("$", " ".join(cmd))
            print(out)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
