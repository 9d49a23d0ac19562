"""Builds the CUDA library libattn.so in-tree with nvcc (sm_103a only), and the
compiled part of its Python binding (_bind.so) with the host compiler.

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
           "vconv.cu", "kv8.cu", "kvp.cu"]
HEADERS = ["ptx.cuh", "attn_internal.h", "bias.cuh", "window.cuh"]

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
    files += [os.path.join(INCLUDE, h) for h in ("attn.h", "ffn.h", "kvcache.h")]
    files.append(BIND_SOURCE)
    return max(os.path.getmtime(f) for f in files)


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


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime()
                         for f in (LIB, BIND)):
        return LIB
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        log = open(os.path.join(BUILD, src.replace(".cu", ".log")), "w")
        cmd = [cc, *ARCH, *FLAGS, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
        objs.append(obj)
    tmp = os.path.join(BUILD, f"_bind.tmp{os.getpid()}.so")
    log = open(os.path.join(BUILD, "bind.log"), "w")
    procs.append(("bind.cpp", subprocess.Popen(_bind_command(tmp), stdout=log,
                                               stderr=subprocess.STDOUT), log))
    failed = []
    for src, pr, log in procs:
        rc = pr.wait()
        log.close()
        if rc != 0:
            failed.append(src)
    if failed:
        msgs = []
        for src in failed:
            with open(os.path.join(BUILD, os.path.splitext(src)[0] + ".log")) as f:
                msgs.append(f"--- {src}\n" + f.read()[-6000:])
        raise RuntimeError("compilation failed:\n" + "\n".join(msgs))
    if verbose:
        for src in SOURCES:
            with open(os.path.join(BUILD, src.replace(".cu", ".log"))) as f:
                print(f.read())
    os.replace(tmp, BIND)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
