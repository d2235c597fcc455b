"""The extension module that marshals the device calls, built here against a stand-in for libmlg
whose calls report how they were called: the module itself, without a GPU."""
import importlib.util
import os
import subprocess
import sysconfig
import threading
import time

import pytest

from lora_moe_expert_gb300 import build

INCLUDE = sysconfig.get_paths()["include"]

# mlg_sort_slots says whether its thread holds the interpreter; mlg_gather_q4 takes n_slots ms.
STAND_IN = r"""
#include <Python.h>
#include <time.h>
#include "mlg.h"
extern "C" {
mlg_status mlg_sort_slots(const int32_t *, const int32_t *, int32_t *, int32_t *, int32_t *, int32_t,
                          int32_t, int32_t, int32_t, void *) { return PyGILState_Check(); }
mlg_status mlg_gather_q4(const mlg_bf16 *, const int32_t *, const uint8_t *, const mlg_bf16 *,
                         const uint8_t *, mlg_bf16 *, int32_t n_slots, int32_t, int32_t, int32_t,
                         int32_t, int32_t, void *) {
  struct timespec t = {n_slots / 1000, n_slots % 1000 * 1000000L};
  nanosleep(&t, nullptr);
  return 0;
}
mlg_status mlg_route_topk(const void *, int32_t, int64_t, int32_t *, float *, int32_t, int32_t,
                          int32_t, int32_t, void *) { return 0; }
mlg_status mlg_route_topk_backward(const void *, int32_t, int64_t, const int32_t *, const float *,
                                   const float *, void *, int64_t, int32_t, int32_t, int32_t,
                                   int32_t, void *) { return 0; }
mlg_status mlg_dispatch(const void *, int32_t, int64_t, const int32_t *, const int32_t *, int32_t *,
                        int32_t *, int32_t *, void *, int32_t, int32_t, int32_t, int32_t, int32_t,
                        void *) { return 0; }
mlg_status mlg_combine(const void *, int32_t, const int32_t *, const float *, void *, int64_t,
                       int32_t, int32_t, int32_t, int32_t, void *) { return 0; }
mlg_status mlg_combine_backward(const void *, int32_t, int64_t, const void *, const int32_t *,
                                const float *, const int32_t *, void *, float *, int32_t, int32_t,
                                int32_t, int32_t, void *) { return 0; }
}
"""


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    if not os.path.exists(os.path.join(INCLUDE, "Python.h")):
        pytest.skip("Python's headers are not installed")
    at = tmp_path_factory.mktemp("extension")
    (at / "stand_in.cpp").write_text(STAND_IN)
    out = at / ("_mlg_py" + sysconfig.get_config_var("EXT_SUFFIX"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE, "-I",
                    build.INCLUDE, os.path.join(build.CSRC, "mlg_py.cpp"), str(at / "stand_in.cpp"),
                    "-o", str(out)], check=True)
    spec = importlib.util.spec_from_file_location("_mlg_py", str(out))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_call_does_not_hold_the_interpreter(module):
    """A launch waits where the stream's queue is full; what would empty it may need Python."""
    assert module.mlg_sort_slots(0, None, 0, 0, 0, 8, 1, 4, 1, 0) == 0


def test_other_threads_run_during_a_call(module):
    ticks = []
    done = threading.Event()

    def count():
        while not done.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.001)

    t = threading.Thread(target=count)
    t.start()
    begin = time.monotonic()
    module.mlg_gather_q4(0, 0, 0, 0, None, 0, 500, 1, 1, 1, 1, 32, 0)
    end = time.monotonic()
    done.set()
    t.join()
    assert sum(begin + 0.1 < at < end - 0.1 for at in ticks) > 3
