"""As many rows as an int32 counts: the norm and its gradient over 2^31 - 1 rows of 16 bytes, in place
(34 GB), whose first, middle and last rows have the bits of a call of their own."""
import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402

pytestmark = pytest.mark.gpu

N, W, SOME = (1 << 31) - 1, 4, 100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("backward", [False, True])
def test_rows_up_to_the_limit_of_int32(backward):
    x = torch.ones(N, W, device="cuda")
    at = [slice(0, SOME), slice(N // 2, N // 2 + SOME), slice(N - SOME, N)]
    rows = torch.randn(len(at) * SOME, W, generator=torch.Generator().manual_seed(0)).cuda()
    for i, s in enumerate(at):
        x[s] = rows[i * SOME:(i + 1) * SOME]
    w = torch.tensor([0.5, 1.0, 1.5, 2.0], device="cuda")
    want = torch.empty_like(rows)
    if backward:  # of a residual sum without branch or norm: dx = 0.75 dout
        mlg.mlg_block_norm_backward(x, None, None, None, None, None, None, x, None, None, None, None,
                                    None, N, W, residual_scale=0.75)
        want = rows * 0.75
    else:
        mlg.mlg_block_norm(x, None, None, None, w, None, x, N, W)
        mlg.mlg_block_norm(rows, None, None, None, w, None, want, len(rows), W)
    for i, s in enumerate(at):
        assert torch.equal(x[s], want[i * SOME:(i + 1) * SOME])
    torch.cuda.synchronize()
