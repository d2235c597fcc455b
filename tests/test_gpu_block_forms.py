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


def test_a_tokens_rows_in_any_batch_where_all_go_call_by_call():
    """The same codes, and the same rows of the experts that both runs chose, bit for bit."""
    block = blk.random_block(2, 12, 272, 144, 3, few_tokens=0)
    x = _x(70, 272, 1)
    kept = []
    for batch in (x, x[:5], x[33:34]):
        block.forward(batch, keep=True)
        kept.append(block.saved)
    for s, first in ((kept[1], 0), (kept[2], 33)):
        T = s["indices"].shape[0]
        mine, other = s["indices"], kept[0]["indices"][first:first + T]
        same = mine == other
        assert same.float().mean() > 0.9  # (the router's products may round a tie apart)
        for name in ("q", "scales", "gate_up", "act_q", "act_scales", "rows"):
            a = s[name].view(torch.uint8)[s["pos"].long()]
            b = kept[0][name].view(torch.uint8)[kept[0]["pos"].long()][3 * first:3 * (first + T)]
            assert torch.equal(a[same.view(-1)], b[same.view(-1)]), name


def test_an_adapter_leaves_tokens_that_do_not_use_it_as_they_were():
    """Two blocks of the same weights, one with adapters, a batch of which every second token uses one."""
    plain, adapted = (blk.random_block(3, 8, 256, 128, 2, rank, few_tokens=0) for rank in (0, 8))
    for name in ("norm_in", "norm_out", "router", "gate_up", "gate_up_scales", "down", "down_scales"):
        setattr(plain, name, getattr(adapted, name))
    x = _x(12, 256, 2)
    row_map = torch.zeros(12, dtype=torch.int32, device="cuda")
    row_map[::2] = -1
    want, _ = plain.forward(x)
    got, _ = adapted.forward(x, row_map=row_map)
    assert torch.equal(got[::2], want[::2]) and not torch.equal(got[1::2], want[1::2])


@pytest.mark.parametrize("few,T,one_call", [(0, 1, False), (4, 4, True), (4, 5, False), (64, 64, True),
                                            (64, 65, False)])
def test_the_form_by_the_tokens(few, T, one_call):
    block = blk.random_block(4, 8, 128, 64, 2, few_tokens=few)
    block.forward(_x(T, 128), keep=True)
    assert ("rows" not in block.saved) == one_call


@pytest.mark.parametrize("few", [-1, 65])
def test_a_limit_that_the_layer_does_not_have_is_refused(few):
    with pytest.raises(ValueError):
        blk.random_block(4, 8, 128, 64, 2, few_tokens=few)
