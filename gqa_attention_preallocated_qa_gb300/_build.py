"""Builds ``libqa.so`` (the C ABI of include/qa.h) in-tree with nvcc for sm_103a,
and beside it ``_q4calls``, the binding's native marshalling of the calls that
are made once per layer and token, under the name that this interpreter gives
its extension modules.  Where g++ or Python's headers are missing the library is
built alone; the binding then lacks those calls.

Each .cu file compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so the library loads
on a machine without a GPU (every CUDA call then fails with a status code).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import threading
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqa.so")
CALLS = os.path.join(PKG, "_q4calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["qa_api.cu", "k1_norm_rope_append.cu", "k2_prefill_tcgen05.cu", "k3_decode_splitkv.cu",
           "q4_api.cu", "k4_q4_rows.cu", "k5_q4_decode.cu",
           "prefill_ws.cu", "q8_api.cu", "k6_q8_rows.cu", "k7_q8_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_lock = threading.Lock()


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqa.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "qa.h"))
    files.append(os.path.abspath(__file__))
    return files


def _cxx() -> str | None:
    return os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")


def can_build_calls() -> bool:
    return bool(_cxx()) and os.path.exists(os.path.join(sysconfig.get_path("include"), "Python.h"))


def stale() -> bool:
    made = [LIB] + ([CALLS] if can_build_calls() else [])
    if not all(os.path.exists(f) for f in made):
        return True
    t = min(os.path.getmtime(f) for f in made)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas", "-v",
           "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC, *extra,
           "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(obj + ".log", "w") as fh:
        fh.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def _build_calls() -> None:
    """_q4calls: plain C++ against this interpreter's headers, no CUDA."""
    if not can_build_calls():
        warnings.warn("g++ or Python.h not found: the binding will lack the 4-bit and 8-bit caches' per-token calls")
        return
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [_cxx(), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-fwrapv",
           "-I", sysconfig.get_path("include"), os.path.join(CSRC, "q4_calls.cpp"), "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on q4_calls.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS)


def build(force: bool = False, extra=()) -> str:
    """Compile and link libqa.so and _q4calls if any source changed (or ``force``)."""
    with _lock:
        if not force and not stale():
            return LIB
        os.makedirs(BUILD, exist_ok=True)
        with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
            calls = ex.submit(_build_calls)
            objs = list(ex.map(lambda s: _compile(s, list(extra)), SOURCES))
            calls.result()
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static",
               "-Xlinker", "--version-script=" + os.path.join(CSRC, "libqa.map"), "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
