"""Builds libmladecode.so in-tree for sm_103a (no cmake; parallel nvcc), and the
CPython module _mla_calls.so that passes torch tensors to it.

    python -m paged_mla_decode_08_gb300.build      # or build() from Python

Objects go to ``_build/`` at the repository root, the library to
``paged_mla_decode_08_gb300/lib/``.  A source-hash stamp skips the build
when nothing changed.
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
                "mla_plan_device.cu", "mla_kv_write.cu", "mla_norm_quant.cu", "mla_gemm_fp8.cu"]
CXX_SOURCES = ["mla_plan.cpp"]
CALLS_SOURCE = "mla_torch_calls.cpp"  # built against this machine's Python and torch
HEADERS = ["mla_internal.h", "per_device.h", "sm103_ptx.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", INCLUDE]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str:
    """torch's folder, without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found")
    return os.path.dirname(spec.origin)


def _stamp() -> str:
    h = hashlib.sha256()
    for f in sorted(CUDA_SOURCES + CXX_SOURCES + HEADERS + [CALLS_SOURCE]):
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    with open(os.path.join(INCLUDE, "mla_decode.h"), "rb") as fh:
        h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + CXX_FLAGS).encode())
    h.update(os.uname().machine.encode())
    h.update((sys.version + importlib.metadata.version("torch") + _torch_dir()).encode())
    return h.hexdigest()


def _run(cmd, log):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if log is not None:
        log.append((cmd, r.stdout))
    if r.returncode != 0:
        raise RuntimeError(f"build step failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}")
    return r.stdout


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA/C++ source and link the shared library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    stamp = _stamp()
    stamp_file = os.path.join(BUILD, "stamp")
    if not force and os.path.exists(LIB) and os.path.exists(CALLS) and os.path.exists(stamp_file):
        with open(stamp_file) as fh:
            if fh.read().strip() == stamp:
                return LIB
    nvcc = _nvcc()
    log: list = []
    jobs = []
    objs = []
    for src in CUDA_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        jobs.append([nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    for src in CXX_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        jobs.append([os.environ.get("CXX", "g++"), *CXX_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    torch_dir, cuda = _torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    cxx, calls_obj = os.environ.get("CXX", "g++"), os.path.join(BUILD, CALLS_SOURCE + ".o")
    jobs.append([cxx, *CXX_FLAGS, "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch_dir, "include"),
                 "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                 "-isystem", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, CALLS_SOURCE), "-o", calls_obj])
    with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
        list(ex.map(lambda c: _run(c, log), jobs))
    tmp = LIB + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], log)
    os.replace(tmp, LIB)
    tmp = CALLS + ".tmp"
    _run([cxx, "-shared", "-o", tmp, calls_obj, "-L" + LIBDIR, "-l:libmladecode.so", "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], log)
    os.replace(tmp, CALLS)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
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
