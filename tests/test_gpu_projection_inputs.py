"""What a projection's caller may hand in: strided activations, tokens without an adapter, empty
batches; and what is refused."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402

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


@pytest.fixture(scope="module")
def proj():
    from lora_moe_expert_gb300.projection import random_projection

    return random_projection(1, 10, 96, 72, 4, 16, 32)


def _batch(p, T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, p.k_in, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, p.n_experts, generator=g, device="cuda").to(torch.bfloat16)
    return x, logits


def _map(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 23])
def test_a_slice_of_wider_activations(proj, T):
    """The columns of a wider tensor, and one token's row repeated: what a contiguous copy gives."""
    x, logits = _batch(proj, T)
    wide = torch.full((T, 3 * proj.k_in), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, proj.k_in:2 * proj.k_in] = x
    row_map = _map([t % 3 - 1 for t in range(T)])
    part = wide[:, proj.k_in:2 * proj.k_in]
    assert torch.equal(proj.decode(part, logits, row_map), proj.decode(x, logits, row_map))
    assert torch.equal(proj.prefill(part, logits), proj.prefill(x, logits))
    same, copies = x[:1].expand(T, -1), x[:1].repeat(T, 1)
    assert torch.equal(proj.decode(same, logits, row_map), proj.decode(copies, logits, row_map))
