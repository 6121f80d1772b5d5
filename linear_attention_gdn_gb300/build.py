"""Build the sm_103a library libgdn.so in-tree (linear_attention_gdn_gb300/_build).

Each .cu under csrc/ compiles to an object in parallel with
    nvcc -gencode arch=compute_103a,code=sm_103a -O3 -lineinfo
and the objects link into one shared library exporting the C ABI of
include/gdn.h.  csrc/gdn_call.c, the binding's argument marshalling, is a Python
extension of its own, named after the interpreter that it is built for.  No torch, no cmake.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
CALL = os.path.join(BUILD, "_gdn_call" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def call_job(force: bool = False):
    """The command that builds the marshalling module, in a list; none where it is up to date, or where this interpreter
    has no headers (the binding then marshals through ctypes).  By nvcc's host compiler, as the library."""
    src, include = os.path.join(CSRC, "gdn_call.c"), sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")) or not (force or _stale(CALL, [src])):
        return []
    return [[NVCC, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "none", "-I", include, src, "-o",
             CALL + f".{os.getpid()}.tmp"]]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([NVCC, *ARCH, *FLAGS, *extra, "-c", s, "-o", o])

    jobs_call = call_job(force)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("failed: " + " ".join(cmd))

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs + jobs_call))
    if jobs_call:
        os.replace(CALL + f".{os.getpid()}.tmp", CALL)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        run([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
