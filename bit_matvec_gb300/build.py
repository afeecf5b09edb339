"""Build libtq.so (the C-ABI library) from csrc/*.cu with nvcc for sm_103a, and the Python
argument marshalling of csrc/tq_call.c with the host compiler.

Each translation unit compiles in parallel; the shared library links the
CUDA runtime statically, so it loads next to any PyTorch build. The output
goes in-tree to bit_matvec_gb300/_lib/libtq.so (git-ignored) and is rebuilt
when a source or header is newer than it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(OUT_DIR, "obj")
LIB = os.path.join(OUT_DIR, "libtq.so")
CALL_SRC = os.path.join(CSRC, "tq_call.c")
CALL = os.path.join(OUT_DIR, "_tq_call.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "tq.h")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + p.stdout)
    return p.stdout


def build_call(force: bool = False) -> str:
    """The extension module that marshals the calls made once or more a decode step."""
    deps = [CALL_SRC, os.path.join(ROOT, "include", "tq.h")]
    if force or _stale(CALL, deps):
        cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
        if not cc:
            raise RuntimeError("no C compiler found (set CC)")
        tmp = CALL + f".tmp{os.getpid()}"
        _run([cc, "-O2", "-std=c11", "-fPIC", "-shared", "-Wall", "-Wextra",
              "-I", sysconfig.get_paths()["include"], CALL_SRC, "-o", tmp])
        os.replace(tmp, CALL)
    return CALL


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    hdrs = headers()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", os.path.join(ROOT, "include")]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    jobs = []
    for src in sources():
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        if force or ptxas_info or _stale(obj, [src] + hdrs):
            jobs.append((src, obj))

    def compile_one(job):
        src, obj = job
        tmp = obj + f".tmp{os.getpid()}"
        out = _run([cc] + flags + ["-c", src, "-o", tmp])
        os.replace(tmp, obj)
        return src, out

    build_call(force)
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 1)) as ex:
            for src, out in ex.map(compile_one, jobs):
                if verbose or ptxas_info:
                    sys.stdout.write(f"== {os.path.basename(src)}\n{out}")

    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in sources()]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        _run([cc] + ARCH + ["-shared", "--cudart", "static", "-o", tmp] + objs
             + ["-lpthread", "-ldl", "-lrt"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
