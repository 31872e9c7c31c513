"""Builds libmoehost.so (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units compile in parallel into moe_decode_host_gb300/_build/, then
link into moe_decode_host_gb300/libmoehost.so with the CUDA runtime linked
statically.  Only nvcc and a host C++ compiler are needed (no torch, no cmake).
csrc/binding.cc becomes the Python extension _decoder_ops (Python's headers, no link to
the library: it is given the addresses it calls), named for the interpreter it was built
with.  Both are written beside their places and moved there when whole, so that a process
that imports them meanwhile finds the one before or the new one.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoehost.so")
BINDING = os.path.join(PKG, "_decoder_ops" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
         "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoehost.so")


def sources() -> list:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run_all(jobs: list, verbose: bool) -> None:
    """Compiler commands, in parallel; the first that failed raises when all have ended."""
    if not jobs:
        return

    def run(cmd):
        return cmd, subprocess.run(cmd, capture_output=True, text=True)

    with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"the compiler failed on {cmd[-3]}")


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "moehost.h"))
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src] + headers) or ptxas_info:
            cmd = [nvcc] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            jobs.append(cmd)

    binding_src, binding_tmp = os.path.join(CSRC, "binding.cc"), BINDING + f".tmp{os.getpid()}"
    stale_binding = _stale(BINDING, [binding_src, os.path.join(ROOT, "include", "moehost.h")])
    if stale_binding:
        cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
        if not cxx:
            raise RuntimeError("a host C++ compiler is required to build _decoder_ops")
        jobs.append([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", sysconfig.get_paths()["include"], "-I",
                     os.path.join(ROOT, "include"), binding_src, "-o", binding_tmp])

    try:
        _run_all(jobs, verbose or ptxas_info)
        if stale_binding:
            os.replace(binding_tmp, BINDING)
    finally:
        if os.path.exists(binding_tmp):
            os.remove(binding_tmp)
    untagged = os.path.join(PKG, "_decoder_ops.so")  # an earlier build's, which any interpreter would load
    if os.path.exists(untagged):
        os.remove(untagged)
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of libmoehost.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
