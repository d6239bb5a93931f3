"""Build the library in-tree: nvcc for sm_103a, objects compiled in parallel.

Produces ``matmul_selection_gb300/_build/libmm_gb300.so`` and, linked to it,
the Python module of the operators' calls, ``_build/mm_fastcall.*.so``, for the
Python that runs this.  That one needs g++ and Python's headers; without them
the package calls through ctypes.  Usable as ``python matmul_selection_gb300/build.py``.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmm_gb300.so")
FASTCALL = os.path.join(BUILD, "mm_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
FASTCALL_SRC = os.path.join(CSRC, "binding", "fastcall.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    out = []
    for d in (CSRC, os.path.join(CSRC, "kernels")):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cpp")):
                out.append(os.path.join(d, f))
    return out


def headers():
    hs = [os.path.join(ROOT, "include", "mm.h")]
    for d in (CSRC, os.path.join(CSRC, "kernels")):
        hs += [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".h", ".cuh"))]
    return hs


def build_id() -> str:
    h = hashlib.sha1()
    for p in sources() + headers() + [FASTCALL_SRC]:
        with open(p, "rb") as f:
            h.update(os.path.basename(p).encode())
            h.update(f.read())
    return h.hexdigest()[:12]


def _compile(src: str, obj: str, bid: str, verbose: bool) -> None:
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-Wall", f"-DMM_BUILD_ID=\"{bid}\"",
           "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    if src.endswith(".cu"):
        cmd[1:1] = ["-Xptxas", "-v"] if verbose else []
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {src}\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr, file=sys.stderr)


def _compile_fastcall() -> None:
    tmp = FASTCALL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
           "-I", sysconfig.get_paths()["include"], FASTCALL_SRC, "-o", tmp,
           "-L", BUILD, "-l:libmm_gb300.so", "-Wl,-rpath,$ORIGIN"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        print(f"mm_fastcall not built, calls go through ctypes: {e}", file=sys.stderr)
        return
    if r.returncode != 0:
        print(f"mm_fastcall not built, calls go through ctypes:\n{r.stdout}\n{r.stderr}", file=sys.stderr)
        return
    os.replace(tmp, FASTCALL)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    bid = build_id()
    stamp = os.path.join(BUILD, "build_id")
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == bid:
                if not os.path.exists(FASTCALL):  # (built with another Python)
                    _compile_fastcall()
                return LIB
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    workers = min(len(srcs), max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(workers) as ex:
        futs = [ex.submit(_compile, s, o, bid, verbose) for s, o in zip(srcs, objs)]
        for f in futs:
            f.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    for f in os.listdir(BUILD):
        if f.startswith("mm_fastcall"):  # (of another build of the library)
            os.remove(os.path.join(BUILD, f))
    _compile_fastcall()
    with open(stamp, "w") as f:
        f.write(bid)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
