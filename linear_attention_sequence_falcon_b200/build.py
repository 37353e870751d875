"""Builds libfalcon.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_quick.<torch>-<python>.so (csrc/quick_layer.cpp, the short way into the layer
operators) with g++ against the torch that is installed.

    python -m linear_attention_sequence_falcon_b200.build [--force]

Objects go to _build/ at the repository root; the shared library lands next
to this file so that it travels with the source tree.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfalcon.so")
# shares the C++ types of one torch and Python, so its name says which
QUICK = os.path.join(PKG, "_quick.%s-%s.so" % (torch.__version__, sys.implementation.cache_tag))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _replaceable(path):
    """Refuses to build a library that this process has loaded: it would go on
    with the old code, whatever is loaded from the new file later."""
    try:
        with open("/proc/self/maps") as maps:
            loaded = any(line.rstrip("\n").removesuffix(" (deleted)").endswith(os.path.realpath(path)) for line in maps)
    except OSError:
        return
    if loaded:
        raise RuntimeError("%s is out of date, and loaded in this process: build before the first call, or in a process "
                           "of its own" % os.path.basename(path))


def build(force: bool = False, verbose: bool = False) -> str:
    lib = build_library(force, verbose)
    build_quick(force, verbose)
    return lib


def build_quick(force: bool = False, verbose: bool = False) -> str:
    """The short way for this torch and Python: rebuilt when its source or the ABI's header changed."""
    import sysconfig
    src = os.path.join(CSRC, "quick_layer.cpp")
    if not force and not _stale(QUICK, [src, os.path.join(INCLUDE, "falcon.h"), os.path.abspath(__file__)]):
        return QUICK
    _replaceable(QUICK)
    base = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_path("include"), os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = QUICK + ".tmp%d" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wno-attributes",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + p for p in inc] +
           [src, "-o", tmp, "-L" + PKG, "-l:libfalcon.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed: " + " ".join(cmd))
    os.replace(tmp, QUICK)
    return QUICK


def build_library(force: bool = False, verbose: bool = False) -> str:
    deps = _deps()
    # the library is also stale when the set of sources changed (one removed)
    manifest = os.path.join(BUILD, "sources.txt")
    listing = "\n".join(os.path.basename(x) for x in _sources())
    try:
        same_sources = open(manifest).read() == listing
    except OSError:
        same_sources = False
    if not force and same_sources and not _stale(LIB, deps + [os.path.abspath(__file__)]):
        return LIB
    _replaceable(LIB)
    os.makedirs(BUILD, exist_ok=True)
    headers = [d for d in deps if not d.endswith(".cu")]
    objs = []
    jobs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([NVCC] + ARCH + FLAGS + ["-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    tmp = LIB + ".tmp%d" % os.getpid()
    run([NVCC] + ARCH + ["-shared", "-o", tmp] + objs)
    os.replace(tmp, LIB)
    with open(manifest, "w") as fh:
        fh.write(listing)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
