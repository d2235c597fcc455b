"""The 4-bit product when its waits run out: it stops fetching and storing, reports the timeout and
returns; the next call is whole again.  No copy is lost: a hook lets the kernel wait for more bytes
than it asked for, so that its own limit (1 s a wait) ends the call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_q4 import Problem, _ids  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    mlg.mlg_read_device_errors(clear=True)
    yield
    torch.cuda.synchronize()
    assert mlg.mlg_read_device_errors(clear=True) == 0


def _run(p, lose):
    """The output, 7 where nothing was written, and the device errors."""
    n_slots, _, n = p.args[:3]
    out = torch.full((n_slots, n), 7.0, dtype=torch.bfloat16, device="cuda")
    mlg.mlg_test_set_knob(mlg.MLG_TEST_Q4_LOSE, lose)
    try:
        mlg.mlg_gather_q4(p.x, p.idx, p.codes, p.scales, p.zeros, out, *p.args)
    finally:
        mlg.mlg_test_set_knob(mlg.MLG_TEST_Q4_LOSE, 0)
    torch.cuda.synchronize()
    return out, mlg.mlg_read_device_errors(clear=True)


# n_slots, top_k, experts, k, n, group, ids: one warp a tile and several, x in shared memory and not,
# one job a CTA and several
@pytest.mark.parametrize("n_slots,top_k,E,k,n,group,kind", [
    (8, 8, 128, 2048, 768, 128, "mixed"), (512, 8, 128, 768, 2048, 32, "mixed"),
    (9, 1, 2, 49152, 40, 128, "mixed"), (1200, 1, 600, 160, 16, 32, "each")])
def test_waits_that_run_out(n_slots, top_k, E, k, n, group, kind):
    ids = np.arange(n_slots) % E if kind == "each" else _ids(n_slots, n_slots, E, kind)
    p = Problem(n_slots + k, n_slots, top_k, E, k, n, group, True, ids)
    want, errors = _run(p, 0)
    assert errors == 0
    held = torch.from_numpy((ids >= 0) & (ids < E)).cuda()
    out, errors = _run(p, 1)
    assert errors == 1  # a wait ran past its limit
    assert (out[held] == 7).all() and (out[~held] == 0).all()
    again, errors = _run(p, 0)
    assert errors == 0 and torch.equal(again, want)
