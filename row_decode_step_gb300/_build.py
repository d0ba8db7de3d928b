"""Compile the CUDA library in-tree for sm_103a (no torch extension machinery).

The library is plain nvcc output: every csrc/*.cu file becomes an object, the
objects are linked into row_decode_step_gb300/libdl_gb300.so.  Objects are
built in parallel and only when their sources changed.  csrc/paged_call.c, the
CPython side of the paged cache's calls, becomes row_decode_step_gb300/_paged_call.<ABI
tag>.so, built for the interpreter that runs this and found by no other.  It takes the host
compiler and Python's own header; where one is missing the library is built without it, and
the paged cache's calls from Python say so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shlex
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdl_gb300.so")
CALL = os.path.join(PKG, "_paged_call" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _call_compiler():
    """The command that compiles csrc/paged_call.c, less its files; None, with a warning, where it cannot be had."""
    cc = shlex.split(os.environ.get("CC") or "gcc")
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    missing = cc[0] if not shutil.which(cc[0]) else header if not os.path.exists(header) else None
    if missing:
        warnings.warn("%s is missing: %s is not built, and the paged cache's calls from Python will not run"
                      % (missing, os.path.basename(CALL)))
        return None
    return cc + ["-O2", "-Wall", "-shared", "-fPIC", "-I", INCLUDE, "-I", os.path.dirname(header)]


def _deps() -> list:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "dl.h")]


def _stale(target: str, sources: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    cc = nvcc()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + deps):
            jobs.append([cc] + ARCH + NVCC_FLAGS + ["-c", s, "-o", o])

    call_src, call_tmp = os.path.join(CSRC, "paged_call.c"), None
    if force or _stale(CALL, [call_src, os.path.join(INCLUDE, "dl.h")]):
        call_cc = _call_compiler()
        if call_cc:
            call_tmp = CALL + ".tmp.%d" % os.getpid()
            jobs.append(call_cc + [call_src, "-o", call_tmp])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiler failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            list(ex.map(run, jobs))
        if call_tmp:
            os.replace(call_tmp, CALL)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        run([cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
