"""Builds libmlg.so in-tree for sm_103a with nvcc (no cmake, no torch extension).

    python -m lora_moe_expert_gb300.build

Each translation unit compiles in parallel to lora_moe_expert_gb300/_build/,
then one nvcc -shared link writes lora_moe_expert_gb300/libmlg.so.  Where
Python's headers are installed, g++ also builds the extension module _mlg_py
(its file named for this interpreter, so that no other loads it), which hands
the binding's device calls to libmlg faster than ctypes does.
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
PY_MODULE = os.path.join(PKG, "_mlg_py" + sysconfig.get_config_var("EXT_SUFFIX"))
PY_SOURCE = "mlg_py.cpp"

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


def _newer(target: str, deps) -> bool:
    """Whether one of deps is newer than the target, or the target is not there."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _python_include() -> str:
    """The folder of Python.h, or "" where it is not installed."""
    include = sysconfig.get_paths()["include"]
    return include if os.path.exists(os.path.join(include, "Python.h")) else ""


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != PY_SOURCE] + _headers()
    if force or _newer(LIBRARY, deps):
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
        tmp = LIBRARY + ".tmp"
        subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIBRARY)
    source = os.path.join(CSRC, PY_SOURCE)
    if force or _newer(PY_MODULE, [LIBRARY, source, *_headers()]):
        _build_py_module(source)
    return LIBRARY


def _build_py_module(source: str) -> None:
    # An older module goes first: where no new one is built, ctypes calls the new library.
    for old in {PY_MODULE, os.path.join(PKG, "_mlg_py.so")}:
        if os.path.exists(old):
            os.remove(old)
    include = _python_include()
    if not include:
        return
    tmp = PY_MODULE + ".tmp"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                    "-I", include, "-I", INCLUDE, source, "-o", tmp,
                    "-L", PKG, "-l:libmlg.so", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, PY_MODULE)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
