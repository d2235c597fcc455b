"""The row stride of a single row, which torch sets as it likes (a transposed column's is 1): through the
extension module, built here against a stand-in whose calls report their stride, and through ctypes."""
import importlib.util
import os
import subprocess
import sysconfig

import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402
from lora_moe_expert_gb300 import build  # noqa: E402
from test_extension_module import INCLUDE, STAND_IN  # noqa: E402

ROWS_F8 = """
extern "C" mlg_status mlg_rows_f8(const void *, int32_t, int64_t ld, const int32_t *, mlg_f8 *, float *,
                                  int32_t, int32_t, int32_t, int32_t, void *) { return ld; }
"""


@pytest.fixture(scope="module")
def stride(tmp_path_factory):
    """tensor -> the stride that a call gets."""
    if not os.path.exists(os.path.join(INCLUDE, "Python.h")):
        pytest.skip("Python's headers are not installed")
    at = tmp_path_factory.mktemp("extension")
    (at / "stand_in.cpp").write_text(STAND_IN + ROWS_F8)
    out = at / ("_mlg_py" + sysconfig.get_config_var("EXT_SUFFIX"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE, "-I",
                    build.INCLUDE, os.path.join(build.CSRC, "mlg_py.cpp"), str(at / "stand_in.cpp"),
                    "-o", str(out)], check=True)
    spec = importlib.util.spec_from_file_location("_mlg_py", str(out))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return lambda t: m.mlg_rows_f8(t, None, None, None, 0, 0, 1, 16, 1, 1, 0)


CASES = {  # tensor, its stride for a call
    "a transposed column": (torch.zeros(32, 1).t(), 32), "rows": (torch.zeros(3, 32), 32),
    "a row of wider ones": (torch.zeros(3, 48)[1:2, :32], 48), "a slice": (torch.zeros(3, 48)[:, :32], 48),
    "a number a row": (torch.zeros(5, 1), 1), "a column": (torch.zeros(5, 7)[:, 2:3], 7),
    "one number": (torch.zeros(1, 1), 1), "of no rows": (torch.zeros(0, 32), 32),
    "the same row again": (torch.zeros(1, 32).expand(4, 32), 0)}


@pytest.mark.parametrize("name", list(CASES))
def test_strides(stride, name):
    t, want = CASES[name]
    assert stride(t) == want
    assert mlg._stride_of(t) == want


def test_rows_that_are_not_adjacent_are_refused(stride):
    for t in (torch.zeros(32, 3).t(), torch.zeros(2, 64)[:, ::2], torch.zeros(1, 64)[:, ::2]):
        with pytest.raises(ValueError):
            stride(t)
        with pytest.raises(ValueError):
            mlg._stride_of(t)
