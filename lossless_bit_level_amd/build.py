"""Build libibp.so (the IBP library), libibp_kv.so (the 8-bit KV page cache)
and libibp_ceiling.so (the gather-copy floor the benchmark measures the IBP
library against) in-tree with hipcc for gfx950, and _ibp_kv.so (libibp_kv's
binding to torch tensors, host code only) with the host compiler.

Usage: python -m lossless_bit_level_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "ibp.hip")
LIB = os.path.join(PKG, "libibp.so")
KV_SRC = os.path.join(PKG, "csrc", "ibp_kv.hip")
KV_LIB = os.path.join(PKG, "libibp_kv.so")
KV_EXT_SRC = os.path.join(PKG, "csrc", "ibp_kv_torch.cpp")
KV_EXT = os.path.join(PKG, "_ibp_kv.so")
CEILING_SRC = os.path.join(PKG, "csrc", "ceiling.hip")
CEILING_LIB = os.path.join(PKG, "libibp_ceiling.so")
INCLUDE = os.path.join(ROOT, "include")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libibp)")


def command(out: str = LIB, extra=(), src: str = SRC) -> list[str]:
    return [hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
            "-Wall", "-I", INCLUDE,
            # packed fp32 instructions are kept out of every kernel
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            *extra, src, "-o", out]


def extension_command(out: str = KV_EXT, src: str = KV_EXT_SRC) -> list[str]:
    """libibp_kv.so has to be built first: the module links to it."""
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
            "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], src, "-o", out,
            "-L", os.path.join(torch_dir, "lib"), "-L", PKG, f"-l:{os.path.basename(KV_LIB)}",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False) -> str:
    """Compile the libraries, side by side (always recompiles; the IBP
    library takes about a minute)."""
    jobs = []
    for src, lib in ((SRC, LIB), (KV_SRC, KV_LIB), (CEILING_SRC, CEILING_LIB)):
        cmd = command(lib + ".tmp", src=src)
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((lib, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                           stderr=subprocess.STDOUT, text=True)))
    failed = []

    def finish(lib, proc):
        out, _ = proc.communicate()
        if proc.returncode != 0:
            sys.stderr.write(out)
            failed.append(os.path.basename(lib))
        else:
            os.replace(lib + ".tmp", lib)

    for lib, proc in jobs:
        finish(lib, proc)
    if not failed:
        cmd = extension_command(KV_EXT + ".tmp")
        if verbose:
            print(" ".join(cmd), flush=True)
        finish(KV_EXT, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                        text=True))
    if failed:
        raise RuntimeError(f"hipcc failed to build {', '.join(failed)}")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
