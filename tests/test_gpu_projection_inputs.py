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


@pytest.mark.parametrize("T,seed", [(1, 0), (9, 1), (40, 2)])
def test_prefill_of_tokens_without_an_adapter(proj, T, seed):
    """A mixed batch gives each token what the batch of its kind gives: with the adapter, or that
    of a projection that has none.  Bit for bit: a row's arithmetic does not depend on its batch."""
    from lora_moe_expert_gb300.projection import MoeProjection

    plain = MoeProjection(proj.w, proj.top_k)
    x, logits = _batch(proj, T, seed)
    values = [(t + seed) % 2 - 1 for t in range(T)]
    out = proj.prefill(x, logits, _map(values))
    with_it, without = proj.prefill(x, logits), plain.prefill(x, logits)
    uses = torch.tensor([v >= 0 for v in values], device="cuda")
    assert torch.equal(out, torch.where(uses[:, None], with_it, without))
    assert not torch.equal(with_it, without)


def test_prefill_and_decode_agree_on_a_mixed_batch():
    """Both forms of the same weights fold the same tokens.  Prefill's weights are the 4-bit ones
    rounded to bf16, and a row is rounded twice in decode, once in prefill, before the one rounding
    of the sum: five roundings of 2^-9 rms at most, independent, so about 0.005 of a token's norm;
    a fold that one form leaves out is most of it."""
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(3, 10, 96, 72, 4, 16, 32)
    x, logits = _batch(p, 24, 3)
    row_map = _map([t % 2 - 1 for t in range(24)])
    a, b = p.prefill(x, logits, row_map).double(), p.decode(x, logits, row_map).double()
    assert ((a - b).norm(dim=1) <= 0.02 * b.norm(dim=1)).all()


def test_an_empty_batch(proj):
    x, logits = _batch(proj, 0)
    row_map = _map([])
    for out in (proj.prefill(x, logits), proj.prefill(x, logits, row_map),
                proj.decode(x, logits, row_map)):
        assert out.shape == (0, proj.n_out) and out.dtype == torch.bfloat16
    dy_rows, dlogits = proj.backward(out)
    assert dy_rows.shape == (0, proj.n_out) and dlogits.shape == (0, proj.n_experts)
    assert proj.rows_backward(torch.empty_like(x)).shape == (0, proj.k_in)


def _refused(error, call, *args):
    with pytest.raises(error):
        call(*args)


def test_refused_batches(proj):
    """What would be read as something else, or past its end."""
    x, logits = _batch(proj, 6)
    row_map = _map([0] * 6)
    for run in (proj.prefill, proj.decode):
        for bad in ((x[:, :-32], logits, row_map), (x, logits[:5], row_map),
                    (x, logits[:, :-1], row_map), (x, logits, row_map[:5]), (x[:5], logits, row_map),
                    (x.cpu(), logits, row_map), (x, logits, row_map.cpu())):
            _refused(ValueError, run, *bad)
        for bad in ((x.float(), logits, row_map), (x, logits, row_map.long()),
                    (x, logits.half(), row_map)):
            _refused(TypeError, run, *bad)


def test_refused_gradients(proj):
    """The gradient of the saved batch, and of no other."""
    x, logits = _batch(proj, 6)
    out = proj.prefill(x, logits)
    dx_rows = torch.zeros(6 * proj.top_k, proj.k_in, dtype=torch.bfloat16, device="cuda")
    for bad in (torch.cat([out, out]), out[:5], out[:, :-8], out.cpu()):
        _refused(ValueError, proj.backward, bad)
    _refused(TypeError, proj.backward, out.float())
    for bad in (torch.cat([dx_rows, dx_rows]), dx_rows[:-1], dx_rows[:, :-8], dx_rows.cpu(),
                torch.cat([dx_rows, dx_rows], 1)[:, :proj.k_in]):
        _refused(ValueError, proj.rows_backward, bad)


def test_refused_weights(proj):
    from lora_moe_expert_gb300.projection import MoeProjection

    codes, scales, zeros, group = proj.q4
    high = zeros.clone()
    high[-1, -1, -1] = 16
    for bad in ((codes[:-1], scales, zeros, group), (codes, scales[:, :, :-1], zeros, group),
                (codes, scales, zeros[:, :-1], group), (codes, scales, high, group),
                (codes, scales, zeros, 2 * group), (codes.cpu(), scales, zeros, group)):
        _refused(ValueError, lambda: MoeProjection(proj.w, 4, q4=bad))
    for bad in ((codes, scales.half(), zeros, group), (codes, scales, zeros.to(scales.dtype), group),
                (codes.to(torch.int8), scales, zeros, group)):
        _refused(TypeError, lambda: MoeProjection(proj.w, 4, q4=bad))
    ids, scale = list(range(0, proj.n_experts, 2)), proj.scale_table[::2].cpu().numpy()
    for bad in ((ids, proj.A[:, :, :-8], proj.B, scale), (ids, proj.A, proj.B[:-1], scale)):
        _refused(ValueError, lambda: MoeProjection(proj.w, 4, lora=bad))
    _refused(TypeError, lambda: MoeProjection(proj.w.half(), 4))
    _refused(TypeError, lambda: MoeProjection(proj.w, 4, lora=(ids, proj.A.float(), proj.B, scale)))


def test_four_bit_weights_in_another_order(proj):
    """Strided 4-bit tensors are laid out once, when the projection is made."""
    from lora_moe_expert_gb300.projection import MoeProjection

    codes, scales, zeros, group = proj.q4
    turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (codes, scales, zeros)]
    x, logits = _batch(proj, 5)
    lora = (list(range(0, proj.n_experts, 2)), proj.A, proj.B, proj.scale_table[::2].cpu().numpy())
    other = MoeProjection(proj.w, proj.top_k, lora=lora, q4=(*turned, group))
    assert torch.equal(other.decode(x, logits, _map([0] * 5)), proj.decode(x, logits, _map([0] * 5)))


def test_nothing_is_kept_without_keep():
    """A serving process holds no rows of its last batch, and has no gradient of it."""
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(2, 10, 96, 72, 4, 16, 32)
    x, logits = _batch(p, 700)
    _refused(RuntimeError, p.backward, x)
    _refused(RuntimeError, p.rows_backward, x)
    kept = p.prefill(x, logits)
    dy_rows, _ = p.backward(kept)
    assert dy_rows.shape == (2800, p.n_out)
    del dy_rows
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out = p.prefill(x, logits, keep=False)
    assert torch.equal(out, kept)
    # the rows of the kept batch are gone, and those of this one
    assert torch.cuda.memory_allocated() - before <= out.numel() * 2 + 512 - 2800 * p.n_out * 2
    _refused(RuntimeError, p.backward, out)
    _refused(RuntimeError, p.rows_backward, x)
