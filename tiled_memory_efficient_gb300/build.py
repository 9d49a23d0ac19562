"""Builds the CUDA library libattn.so in-tree with nvcc (sm_103a only), and the
compiled part of its Python binding (_bind.so) with the host compiler where torch is
installed.

    python -m tiled_memory_efficient_gb300.build [--force]

Each .cu file compiles in parallel to an object file under _build/, then one
link step produces _build/libattn.so against the shared CUDA runtime.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libattn.so")
BIND = os.path.join(BUILD, "_bind.so")
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

SOURCES = ["abi.cu", "attn_fwd.cu", "attn_bwd.cu", "bwd_noalloc.cu", "splitkv.cu", "ffn.cu",
           "vconv.cu", "kv8.cu", "kvp.cu", "rope.cu", "kv8_shared.cu",
           "kv8_shared_attn.cu"]
HEADERS = ["ptx.cuh", "attn_internal.h", "bias.cuh", "window.cuh", "kv8.cuh", "kv8_attn.cuh", "rope.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    return max(os.path.getmtime(f) for f in files + _public_headers())


def _public_headers() -> list:
    return [os.path.join(INCLUDE, h) for h in ("attn.h", "ffn.h", "kvcache.h", "rope.h")]


def _have_torch() -> bool:
    import importlib.util
    return importlib.util.find_spec("torch") is not None


def _bind_command(out: str) -> list:
    """Compiles and links bind.cpp against the installed torch and Python."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for i in inc for x in ("-isystem", i)], BIND_SOURCE, "-o", out,
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _start(src: str, cmd: list):
    """A compiler process whose output goes to the log of `src`."""
    log = open(os.path.join(BUILD, os.path.splitext(src)[0] + ".log"), "w")
    with log:
        return src, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)


def _finish(procs: list) -> None:
    failed = [src for src, pr in procs if pr.wait() != 0]
    if failed:
        msgs = []
        for src in failed:
            with open(os.path.join(BUILD, os.path.splitext(src)[0] + ".log")) as f:
                msgs.append(f"--- {src}\n" + f.read()[-6000:])
        raise RuntimeError("compilation failed:\n" + "\n".join(msgs))


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is out of date: the library, which needs nvcc alone, and beside it the
    compiled part of the Python binding where torch is installed."""
    os.makedirs(BUILD, exist_ok=True)
    stale = lambda f, newest: force or not os.path.exists(f) or os.path.getmtime(f) < newest
    bind, tmp_bind = [], BIND + f".tmp{os.getpid()}"
    if _have_torch() and stale(BIND, max(os.path.getmtime(f) for f in [BIND_SOURCE] + _public_headers())):
        bind = [_start("bind.cpp", _bind_command(tmp_bind))]
    try:
        if stale(LIB, _deps_mtime()):
            _build_library(verbose)
    finally:
        _finish(bind)
    if bind:
        os.replace(tmp_bind, BIND)
    return LIB


def _build_library(verbose: bool) -> None:
    cc = nvcc()
    objs = [os.path.join(BUILD, src.replace(".cu", ".o")) for src in SOURCES]
    _finish([_start(src, [cc, *ARCH, *FLAGS, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj])
             for src, obj in zip(SOURCES, objs)])
    if verbose:
        for src in SOURCES:
            with open(os.path.join(BUILD, src.replace(".cu", ".log"))) as f:
                print(f.read())
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
