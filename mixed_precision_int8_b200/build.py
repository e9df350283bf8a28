"""Build the sm_100a CUDA library libllmint8.so in-tree with nvcc.

The library exposes only the C ABI of include/llmint8.h. It is compiled for
sm_100a alone (tcgen05 / TMA code has no other target) with IEEE division
(no fast math), which the bit-exact quantisation relies on.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libllmint8.so")
SOURCES = [os.path.join(CSRC, f) for f in ("llmint8_api.cu", "finetune_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith(".cuh")] + [os.path.join(INCLUDE, "llmint8.h")]


def nvcc_path() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def nvcc_flags(verbose_ptxas: bool = False):
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
             "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    return flags


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(d) for d in DEPS)):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    nvcc = [nvcc_path()] + nvcc_flags(verbose_ptxas)
    objs = [f"{tmp}.{os.path.basename(s)}.o" for s in SOURCES]
    try:
        # one compiler per source file, all at once
        procs = [subprocess.Popen(nvcc + ["-c", "-o", o, s]) for s, o in zip(SOURCES, objs)]
        for p in [p for p in procs if p.wait() != 0]:
            raise subprocess.CalledProcessError(p.returncode, p.args)
        subprocess.run(nvcc + ["-shared", "-o", tmp] + objs, check=True)
        os.replace(tmp, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
