"""A decode step right after kernels that rewrite the adapter.  The decode fold reads its tables and
pairs before the kernel ahead of it has completed; that kernel is the 4-bit product, which lets it
start only after everything before itself is written.  So a projection's adapter can be rotated by
kernels of the same stream, without the fold's flag for a preceding writer."""
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


@pytest.mark.parametrize("what", ["pairs", "tables"])
@pytest.mark.parametrize("n_experts,k_in,n_out,rank,T", [(96, 768, 2048, 16, 16), (24, 1024, 256, 64, 1),
                                                         (128, 768, 2048, 32, 64)])
def test_decode_after_kernels_that_rewrite_the_adapter(n_experts, k_in, n_out, rank, T, what):
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(1, n_experts, k_in, n_out, 4, rank, 128)
    x = torch.randn(T, k_in, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, n_experts, device="cuda").to(torch.bfloat16)
    row_map = torch.zeros(T, dtype=torch.int32, device="cuda")
    # the adapters to turn between: other pairs in the same place, or other places
    pairs = [(p.A.clone(), p.B.clone())] + [
        (torch.randn_like(p.A) / k_in ** 0.5, torch.randn_like(p.B) / rank ** 0.5) for _ in range(2)]
    step_a, step_b = p.A[0].numel() * 2, p.B[0].numel() * 2
    tables = []
    for A, B in pairs:
        i = torch.arange(len(A), device="cuda")
        a, b = torch.zeros_like(p.a_table), torch.zeros_like(p.b_table)
        a[::2], b[::2] = A.data_ptr() + i * step_a, B.data_ptr() + i * step_b
        tables.append((a, b))

    def rotate(i):
        if what == "pairs":
            torch.mul(pairs[i][0], 1.0, out=p.A)
            torch.mul(pairs[i][1], 1.0, out=p.B)
        else:
            torch.bitwise_or(tables[i][0], 0, out=p.a_table)
            torch.bitwise_or(tables[i][1], 0, out=p.b_table)

    want = []
    for i in range(3):
        rotate(i)
        torch.cuda.synchronize()
        want.append(p.decode(x, logits, row_map))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = []
    for i in range(60):
        rotate(i % 3)
        got.append(p.decode(x, logits, row_map))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 3]), i
