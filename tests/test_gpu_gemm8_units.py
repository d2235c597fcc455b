"""The e4m3 expert product where a CTA takes several units one after the other, in short sums over
full tiles: result boxes used again, also after columns that n_out cuts off, both accumulators across
units, scales asked for a unit ahead."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_rows_f8 import _codes, _counts, _scales  # noqa: E402

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


def _check(offsets, rows, k, n, experts):
    """Six runs, each into an out of its own: the bits of the first, which is within the bound."""
    x, xs = _codes((rows, k), 1), _scales((rows, refs.blocks(k)), 2)
    w, ws = _codes((experts, n, k), 3), _scales((experts, refs.blocks(n), refs.blocks(k)), 4)
    outs = [torch.full((rows, n), -3.0, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    for out in outs:
        mlg.mlg_grouped_gemm_f8(x, xs, offsets, w, ws, out, rows, k, n, experts)
    spans = [0, rows] if offsets is None else offsets.tolist()
    for e, (lo, hi) in enumerate(zip(spans, spans[1:])):
        if lo < hi:
            ref, err = refs.gemm_f8(x[lo:hi].double().cpu().numpy(), xs[lo:hi].cpu().numpy(),
                                    w[e].double().cpu().numpy(), ws[e].cpu().numpy())
            operator_refs.assert_within(outs[0][lo:hi].double().cpu().numpy(), ref, err, True,
                                        f"expert {e}")
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


# n: a half of 128 columns that ends after one, two or three boxes of 32, alone, beside a whole half
# and in a second chunk of 256; n of 8 ends inside a box
@pytest.mark.parametrize("k", [16, 128, 400])
@pytest.mark.parametrize("n", [8, 32, 64, 96, 128, 160, 288, 360])
def test_dense(n, k):
    _check(None, 612 * 128 + 45, k, n, 1)  # at least four units a CTA


@pytest.mark.parametrize("experts,rows,k,n", [(40, 60000, 144, 96), (40, 60000, 144, 328),
                                              (300, 70001, 272, 200), (3, 50000, 1024, 64)])
def test_experts(experts, rows, k, n):
    """Whole and partial tiles mixed."""
    offsets = torch.zeros(experts + 1, dtype=torch.int32)
    offsets[1:] = torch.from_numpy(np.cumsum(_counts("skew", experts, rows, rows)))
    _check(offsets.cuda(), rows, k, n, experts)
