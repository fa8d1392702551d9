"""Build libasffn.so in-tree with nvcc for sm_100a (B200).

Usage: python -m activation_sparse_ffn_predict_b200.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libasffn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("asffn.cu", "w4.cu", "attention.cu", "score.cu", "rotary.cu", "evict.cu",
                                              "lora.cu")]
HEADERS = [os.path.join(CSRC, "common.cuh"), os.path.join(CSRC, "host.cuh"), os.path.join(CSRC, "paged.cuh"), os.path.join(CSRC, "attn.cuh"),
           os.path.join(INCLUDE, "asffn.h")]
DEPS = SOURCES + HEADERS


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libasffn.so")


def flags() -> list:
    return ["-O3", "-std=c++17", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def object_of(source: str) -> str:
    return os.path.splitext(source)[0] + ".o"


def compile_command(source: str, ptxas_verbose: bool = False) -> list:
    return [nvcc_path()] + (["-Xptxas=-v"] if ptxas_verbose else []) + flags() + ["-c", source, "-o",
                                                                                   object_of(source)]


def link_command(out: str = LIB) -> list:
    return [nvcc_path()] + flags() + ["-shared", "-o", out] + [object_of(p) for p in SOURCES]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in DEPS)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    """Compile the stale sources (all with force), side by side, and link."""
    if not force and not ptxas_verbose and up_to_date():
        return LIB
    newest = max(os.path.getmtime(p) for p in HEADERS)
    stale = [p for p in SOURCES if force or ptxas_verbose or not os.path.exists(object_of(p))
             or os.path.getmtime(object_of(p)) < max(newest, os.path.getmtime(p))]
    running = [subprocess.Popen(compile_command(p, ptxas_verbose), stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                text=True) for p in stale]
    said = [p.communicate()[0] for p in running]
    for p, out in zip(running, said):
        if p.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + out)
    tmp = LIB + ".tmp"
    res = subprocess.run(link_command(tmp), capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)
    if not quiet or ptxas_verbose:
        sys.stdout.write("".join(said) + res.stdout + res.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="--ptxas-verbose" in sys.argv, quiet=False)
    print(LIB)
