"""The e4m3 product and the layer of a few tokens when their waits run out: they stop fetching, report
the timeout and return, with outputs that say so; the next call is whole again.  No copy is lost: a hook
lets the kernels wait for more bytes than they asked for, so that their own limit (1 s a wait) ends the
call."""
import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_moe_layer import Layer  # noqa: E402
from test_gpu_rows_f8 import _codes, _scales  # noqa: E402

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


def _errors(call, lose):
    mlg.mlg_test_set_knob(mlg.MLG_TEST_BLOCK_LOSE, lose)
    try:
        call()
    finally:
        mlg.mlg_test_set_knob(mlg.MLG_TEST_BLOCK_LOSE, 0)
    torch.cuda.synchronize()
    return mlg.mlg_read_device_errors(clear=True)


# one unit a CTA and several, both plans (short sums over full tiles, others)
@pytest.mark.parametrize("rows,k,n", [(5, 256, 264), (90000, 144, 96), (40000, 2064, 264)])
def test_product(rows, k, n):
    x, xs = _codes((rows, k), 1), _scales((rows, -(-k // 128)), 2)
    w, ws = _codes((1, n, k), 3), _scales((1, -(-n // 128), -(-k // 128)), 4)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    call = lambda: mlg.mlg_grouped_gemm_f8(x, xs, None, w, ws, out, rows, k, n, 1)  # noqa: E731
    assert _errors(call, 0) == 0
    want = out.clone()
    out.fill_(7.0)
    assert _errors(call, 1) == 1  # a wait ran past its limit
    assert (out == 7).all()
    assert _errors(call, 0) == 0 and torch.equal(out, want)


# few stages and many, a unit a CTA and several, shared k, tokens without a choice
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,E,K,H,inter", [(1, 8, 2, 64, 32), (1, 2, 1, 80, 2064), (43, 97, 6, 1040, 48)])
def test_layer(T, E, K, H, inter, f8):
    layer = Layer(T, E, K, H, inter, f8, T + E, logits="f32")
    if T > 1:
        layer.logits[3] = float("-inf")
    assert _errors(layer.run, 0) == 0
    want = layer.out.clone()
    assert _errors(layer.run, 1) == 1
    held = torch.ones(T, dtype=torch.bool, device="cuda")
    if T > 1:
        held[3] = False
    assert layer.out[:T][held].isnan().all() and not layer.out[:T][~held].any()
    assert (layer.out[T] == 77).all()
    assert _errors(layer.run, 0) == 0 and torch.equal(layer.out, want)
