"""The gated activation over the whole range of its gates, and blocks with an infinity."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lo,hi", [(-88.72, -87.2), (-87.5, -80.0), (-80.0, -1.0), (-1.0, 1.0),
                                   (1.0, 1e4)])
def test_gates(lo, hi, dtype):
    """Within 12 u of the activation (block_refs), and what rounding the reciprocal, a number below
    2^-126, to a multiple of 2^-149 makes of it: |g| 2^-150.  From -88.73 down exp(-g) is infinite."""
    n, inter = 8, 512
    g = torch.Generator().manual_seed(0)
    gate = torch.linspace(lo, hi, n * inter, dtype=torch.float64).view(n, inter)
    up = torch.randn(n, inter, generator=g) * (1e30 if hi < -1 else 1.0)
    v = torch.cat([gate.float(), up], 1).to(dtype)
    v[:, :inter] = v[:, :inter].clamp(min=-88.5 if dtype == torch.bfloat16 else lo)
    act, q = torch.empty(n, inter, dtype=dtype, device="cuda"), torch.empty(n, inter, dtype=F8,
                                                                             device="cuda")
    s = torch.empty(n, inter // 128, device="cuda")
    mlg.mlg_swiglu_f8(v.cuda(), act, q, s, n, inter)
    gate, up = np.split(v.double().numpy(), 2, axis=1)
    a = gate / (1 + np.exp(-gate)) * up
    err = refs.ACT_REL * np.abs(a) + 1.01 * np.abs(gate) * 2.0 ** -150 * np.abs(up)
    operator_refs.assert_within(act.double().cpu().numpy(), a, err, dtype == torch.bfloat16, "act")
    each = refs.spread(s.double().cpu().numpy(), inter, 1)
    half = np.maximum(np.abs(a) * 2.0 ** -4, each * 2.0 ** -10) + err + 2 * refs.U * np.abs(a)
    assert (np.abs(q.double().cpu().numpy() * each - a) <= half).all()


def test_gates_whose_power_leaves_the_range():
    gate = torch.tensor([-88.73, -89.0, -128.0, -1e4, -3e38, 3e38, 0.0, -0.0]).repeat(1, 2)
    v = torch.cat([gate, torch.ones(1, 16)], 1).cuda()
    act = torch.empty(1, 16, device="cuda")
    mlg.mlg_swiglu_f8(v, act, None, None, 1, 16)
    want = torch.where(gate > 0, gate, torch.zeros(()))
    assert torch.equal(act.cpu(), want)


def test_a_block_with_an_infinity_has_nan_codes_alone():
    x = torch.randn(2, 384, generator=torch.Generator().manual_seed(1))
    x[0, 130], x[1, 300] = float("inf"), float("-inf")
    x[0, 128:144] = torch.where(x[0, 128:144].isinf(), x[0, 128:144], torch.zeros(()))
    q, s = torch.empty(2, 384, dtype=F8, device="cuda"), torch.empty(2, 3, device="cuda")
    mlg.mlg_rows_f8(x.cuda(), None, q, s, 2, 384, 1, 2)
    nan = (q.view(torch.uint8) & 0x7f == 0x7f).cpu()
    want = torch.zeros(2, 384, dtype=torch.bool)
    want[0, 128:256], want[1, 256:] = True, True
    assert torch.equal(nan, want)
    assert torch.equal(s.isinf().cpu(), torch.tensor([[False, True, False], [False, False, True]]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1.0, 1e-25, 1e-37, 0.0])
def test_zeros_keep_their_sign(dtype, size):
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(2)) * size
    x[:, ::3], x[:, 1::3] = 0.0, -0.0
    x = x.to(dtype)
    q, s = torch.empty(3, 256, dtype=F8, device="cuda"), torch.empty(3, 2, device="cuda")
    mlg.mlg_rows_f8(x.cuda(), None, q, s, 3, 256, 1, 3)
    each = torch.from_numpy(refs.spread(refs.scales_f32(x.float().numpy()), 256, 1).copy())
    want = (x.float() / each).clamp(-448, 448).to(F8)
    assert torch.equal(q.view(torch.uint8).cpu(), want.view(torch.uint8))
    assert (q.view(torch.uint8)[:, 1::3] == 0x80).all()
