"""What a block keeps of a step, and which form a batch takes."""
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402
from lora_moe_expert_gb300 import block as blk  # noqa: E402

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


def _x(T, hidden, seed=0):
    return torch.randn(T, hidden, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T,rank", [(9, 0), (9, 8), (70, 0), (70, 8)])
def test_saved_activations_are_activations_or_not_there(T, rank):
    block = blk.random_block(1, 8, 256, 144, 2, rank)
    block.forward(_x(T, 256), keep=True)
    s = block.saved
    if s.get("act") is None:
        assert rank == 0
        return
    a, err = refs.swiglu(s["gate_up"].double().cpu().numpy())
    operator_refs.assert_within(s["act"].double().cpu().numpy(), a, err, True)
