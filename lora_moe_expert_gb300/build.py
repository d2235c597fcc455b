"""Builds libmlg.so in-tree for sm_103a with nvcc (no cmake, no torch extension).

    python -m lora_moe_expert_gb300.build

Each translation unit compiles in parallel to lora_moe_expert_gb300/_build/,
then one nvcc -shared link writes lora_moe_expert_gb300/libmlg.so.  Where
Python's headers are installed, g++ also builds _mlg_py.so, which hands the
binding's device calls to libmlg faster than ctypes does.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBRARY = os.path.join(PKG, "libmlg.so")
PY_MODULE = os.path.join(PKG, "_mlg_py.so")

SOURCES = ["mlg_host.cpp", "mlg_gather.cu", "mlg_decode.cu", "mlg_grouped.cu", "mlg_gemm_fold.cu",
           "mlg_route.cu", "mlg_rows.cu", "mlg_q4.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC, "-c",
           os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd[4:4] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    return obj


def _stale(objs) -> bool:
    if not os.path.exists(LIBRARY) or not os.path.exists(PY_MODULE):
        return True
    t = os.path.getmtime(LIBRARY)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "mlg.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and not _stale(SOURCES):
        return LIBRARY
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIBRARY + ".tmp"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIBRARY)
    _build_py_module()
    return LIBRARY


def _build_py_module() -> None:
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return  # the binding then calls through ctypes
    tmp = PY_MODULE + ".tmp"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                    "-I", include, "-I", INCLUDE, os.path.join(CSRC, "mlg_py.cpp"), "-o", tmp,
                    "-L", PKG, "-l:libmlg.so", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, PY_MODULE)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
