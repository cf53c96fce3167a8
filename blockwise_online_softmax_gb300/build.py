"""Build ``libra.so`` in-tree with nvcc, for sm_103a only, and the extension
``_serve.so`` that marshals the serving calls' tensors into it.

Each translation unit is compiled in parallel into ``_build/``.  The
objects are then linked into ``blockwise_online_softmax_gb300/libra.so``
with the CUDA runtime linked statically, so the library needs only the
driver at run time.  ``_serve.so`` is a CPython extension (g++, torch's
headers) linked to it.  Run ``python -m blockwise_online_softmax_gb300.build``
or call ``build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libra.so")
SERVE = os.path.join(PKG, "_serve.so")
SERVE_SOURCE = "serve_binding.cpp"
SOURCES = ["ra_api.cu", "state_kernels.cu", "simt_kernel.cu", "umma_kernel.cu", "decode_kernel.cu",
           "bwd_kernel.cu", "serve_api.cu", "rope_kernel.cu", "pages_kernel.cu",
           "paged_kernel.cu", "paged_tc_kernel.cu", "paged_read_kernel.cu",
           "paged_fp8_kernel.cu", "paged_prefix_kernel.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libra.so")
    return cand


def _flags(extra=()):
    return (ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I" + INCLUDE, "-I" + CSRC] + list(extra))


def _serve_flags():
    """Compile and link flags of the extension: torch as it is installed."""
    import torch

    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(t, "lib")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return (["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}"]
            + [f"-I{i}" if i == INCLUDE else f"-isystem{i}" for i in inc],
            ["-L" + PKG, "-lra", "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
             "-ltorch_cuda", "-lc10_cuda",
             "-Wl,-rpath,$ORIGIN:" + lib])


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(SERVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(SERVE))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "ra.h"),
                                                               os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libra.so; returns its path.  Raises on failure."""
    if not force and not ptxas_info and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    cflags, ldflags = _serve_flags()
    serve_obj = os.path.join(BUILD_DIR, "serve_binding.o")
    procs = [(SERVE_SOURCE, None, subprocess.Popen(
        ["g++"] + cflags + ["-c", os.path.join(CSRC, SERVE_SOURCE), "-o", serve_obj],
        stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))]
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc()] + _flags(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))
    objs, errors = [], []
    for src, obj, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append(f"--- {src} ---\n{out}")
        elif out and (verbose or ptxas_info):
            print(f"--- {src} ---\n{out}", flush=True)
        if obj:
            objs.append(obj)
    if errors:
        raise RuntimeError("compilation failed:\n" + "\n".join(errors))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout)
    os.replace(tmp, LIB)
    tmp = SERVE + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, serve_obj] + ldflags, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the extension failed:\n" + r.stdout)
    os.replace(tmp, SERVE)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
