"""Builds libwq4.so in-tree with nvcc for sm_103a (one object per .cu, compiled in parallel) and, where
torch with CUDA and Python's headers are installed, _wq4_binding.so, which marshals some of its Python calls.

With --debug it builds libwq4_debug.so instead: the same sources with -DWQ4_DEBUG=1, whose kernels
check every copy coordinate, weight record range, scheduled tile and output column before use
(csrc/wq4_check.h) and report a violation as WQ4_ERR_BOUNDS.

Usage: python -m weight_only_quantized_wq4_gb300.builder [--force] [--debug]
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwq4.so")
DEBUG_LIB = os.path.join(PKG, "libwq4_debug.so")
BINDING = os.path.join(PKG, "_wq4_binding.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stamp(flags) -> str:
    h = hashlib.sha256()
    h.update(" ".join(ARCH + flags).encode())
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            if f.endswith(".cpp"):
                continue                          # (the binding: built and stamped by itself)
            with open(os.path.join(d, f), "rb") as fh:
                h.update(f.encode())
                h.update(fh.read())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def _binding_command():
    """The compiler call that makes _wq4_binding.so, or None without what it is made against: torch (found,
    not imported) with CUDA, and Python's headers."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    root = spec.submodule_search_locations[0]
    lib = os.path.join(root, "lib")
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(lib, "libc10_cuda.so")) or not os.path.exists(os.path.join(python, "Python.h")):
        return None
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-I", INCLUDE,
            "-I", python, "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
            os.path.join(CSRC, "wq4_binding.cpp"), "-o", BINDING + ".tmp", "-L" + lib, "-Wl,-rpath," + lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _binding_stamp() -> str:
    """What the binding is made from: its source, the header, and torch's version."""
    h = hashlib.sha256(os.uname().machine.encode())
    files = [os.path.join(CSRC, "wq4_binding.cpp"), os.path.join(INCLUDE, "wq4.h")]
    spec = importlib.util.find_spec("torch")
    if spec is not None and spec.submodule_search_locations:
        files.append(os.path.join(spec.submodule_search_locations[0], "version.py"))
    for f in files:
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _build_binding(stamp: str) -> None:
    cmd = _binding_command()
    if cmd is None:
        return
    stamp = hashlib.sha256((stamp + " ".join(cmd)).encode()).hexdigest()   # (names the Python and torch it is for)
    stamp_file = os.path.join(BUILD, "binding_stamp")
    if os.path.exists(BINDING) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for wq4_binding.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(BINDING + ".tmp", BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp_file, "w") as f:
        f.write(stamp)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile and link the library (the bounds-checking one with debug=True) if sources changed;
    returns the .so path."""
    lib = DEBUG_LIB if debug else LIB
    bdir = os.path.join(BUILD, "debug") if debug else BUILD
    flags = FLAGS + ["-DWQ4_DEBUG=1"] if debug else FLAGS
    stamp = _stamp(flags)
    stamp_file = os.path.join(bdir, "stamp")
    if not force and os.path.exists(lib) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                _build_binding(_binding_stamp())
                return lib
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    workers = min(len(srcs) + 1, max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(workers) as ex:
        binding = ex.submit(_build_binding, _binding_stamp())
        objs = list(ex.map(compile_one, srcs))
        binding.result()
    tmp = lib + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
