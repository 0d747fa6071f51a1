"""Build libpagedkv.so in-tree with nvcc for sm_103a.

    python -m paged_kv_cache_316_gb300.build [--force] [--ptxas-verbose] [--debug-bounds | --all]

Each translation unit under csrc/ is compiled in parallel to an object in
_build/, then linked into paged_kv_cache_316_gb300/libpagedkv.so with the
CUDA runtime linked statically (the library needs no libcudart at load time
and no libcuda at link time).  The debug variant, libpagedkv_debug.so
(objects in _build/debug/), is the same source compiled with
-DPKV_DEBUG_BOUNDS=1: every offset the kernels derive is range-checked
before use (the PKV_DEV_ERR_BOUNDS bit of the error word).

_calls.so, the part of the Python binding that is C++ (csrc/calls.cpp), is
compiled beside them with g++ against the installed torch's headers.  Its name
carries the interpreter's ABI tag, it refuses to be imported under another
torch, and it is compiled again when the command that made it (torch's version
and paths, the flags) changes.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
LIB_DEBUG = os.path.join(HERE, "libpagedkv_debug.so")
LIB_CALLS = os.path.join(HERE, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CALLS_STAMP = os.path.join(BUILD, "calls.stamp")  # the command that made it
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _variant(debug_bounds: bool):
    """(object folder, library path, extra nvcc flags) of one build."""
    if debug_bounds:
        return os.path.join(BUILD, "debug"), LIB_DEBUG, ["-DPKV_DEBUG_BOUNDS=1"]
    return BUILD, LIB, []


def _start(debug_bounds: bool, force: bool, ptxas_verbose: bool):
    """Start the nvcc jobs of one variant; returns (objects, library, jobs)."""
    obj_dir, lib, extra = _variant(debug_bounds)
    os.makedirs(obj_dir, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "pagedkv.h"))
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_verbose or _stale(obj, [src] + headers):
            cmd = [nvcc()] + ARCH + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    return objs, lib, procs


def _finish(objs, lib, procs, force: bool, ptxas_verbose: bool, quiet: bool) -> str:
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            failed.append((src, out))
        elif out and (ptxas_verbose or not quiet):
            sys.stdout.write(out)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    if force or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        subprocess.run([nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs,
                       check=True)
        os.replace(tmp, lib)
    return lib


def _start_calls(force: bool):
    """Start the compilation of _calls.so if it is stale; returns the jobs of
    _finish_calls."""
    import torch
    src = os.path.join(CSRC, "calls.cpp")
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    lib = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPKV_TORCH_VERSION="{torch.__version__}"',
           "-I", INCLUDE, "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src, "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    stamp = "\n".join(cmd)
    if not (force or _stale(LIB_CALLS, [src, os.path.join(INCLUDE, "pagedkv.h")]) or _text(CALLS_STAMP) != stamp):
        return []
    tmp = LIB_CALLS + f".tmp{os.getpid()}"
    pr = subprocess.Popen(cmd + ["-o", tmp], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    return [(src, pr, tmp, stamp)]


def _text(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _finish_calls(jobs):
    for src, pr, tmp, stamp in jobs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            raise RuntimeError(f"g++ failed:\n--- {src}\n{out}")
        os.replace(tmp, LIB_CALLS)
        os.makedirs(BUILD, exist_ok=True)
        with open(CALLS_STAMP, "w") as f:
            f.write(stamp)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True,
          debug_bounds: bool = False) -> str:
    """Build one variant: libpagedkv.so, or with debug_bounds the range-checking
    libpagedkv_debug.so (-DPKV_DEBUG_BOUNDS=1); returns its path."""
    calls = _start_calls(force)
    objs, lib, procs = _start(debug_bounds, force, ptxas_verbose)
    lib = _finish(objs, lib, procs, force, ptxas_verbose, quiet)
    _finish_calls(calls)
    return lib


def build_all(force: bool = False, quiet: bool = True):
    """Build both variants, all translation units compiled in parallel;
    returns (release library, debug library)."""
    calls = _start_calls(force)
    jobs = [_start(d, force, False) for d in (False, True)]
    libs = tuple(_finish(*j, force, False, quiet) for j in jobs)
    _finish_calls(calls)
    return libs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    ap.add_argument("--debug-bounds", action="store_true", help="build libpagedkv_debug.so only")
    ap.add_argument("--all", action="store_true", help="build both libraries")
    a = ap.parse_args()
    if a.all:
        print("\n".join(build_all(force=a.force, quiet=False)))
    else:
        print(build(force=a.force, ptxas_verbose=a.ptxas_verbose, quiet=False,
                    debug_bounds=a.debug_bounds))


if __name__ == "__main__":
    main()
