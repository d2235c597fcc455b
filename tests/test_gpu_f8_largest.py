"""Rows in e4m3 whose width is the most that an int32 counts, and products with the longest k and the
most columns that are taken."""
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
WIDE = (1 << 31) - 16
CUT = WIDE // 256 * 256 - 4096  # what is compared begins here, on a block's boundary


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    mlg.mlg_read_device_errors(clear=True)
    yield
    torch.cuda.synchronize()
    assert mlg.mlg_read_device_errors(clear=True) == 0
    torch.cuda.empty_cache()


def _new(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _zeros(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(F8)


@pytest.mark.parametrize("op", ["rows", "swiglu"])
def test_wide_rows(op):
    halves = 1 if op == "rows" else 2
    x = torch.zeros(1, halves * WIDE, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(0)
    for h in range(halves):
        x[0, h * WIDE + CUT:(h + 1) * WIDE] = torch.randn(WIDE - CUT, generator=g).cuda()
    tail = torch.cat([x[:, h * WIDE + CUT:(h + 1) * WIDE] for h in range(halves)], 1)
    got = []
    for v, width in ((x, WIDE), (tail, WIDE - CUT)):
        q, s = _new(1, width, dtype=F8), _new(1, -(-width // 128), dtype=torch.float32)
        if op == "rows":
            mlg.mlg_rows_f8(v, None, q, s, 1, width, 1, 1)
        else:
            mlg.mlg_swiglu_f8(v, None, q, s, 1, width)
        got.append((q.view(torch.uint8), s))
    (q, s), (tail_q, tail_s) = got
    assert torch.equal(q[:, CUT:], tail_q) and torch.equal(s[:, CUT // 128:], tail_s)
    assert tail_q.any() and not q[:, :CUT].any() and (s[:, :CUT // 128] == 2.0 ** -126).all()


def _codes(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(F8).cuda()


def test_long_sums():
    """Values at the first, some middle and the last codes of k: their products' sum, exactly."""
    k, n = mlg.MLG_F8_MAX_WIDTH, 264
    x, w = _zeros(2, k), _zeros(1, n, k)
    g = torch.Generator().manual_seed(1)
    parts = [slice(0, 96), slice(k // 2, k // 2 + 32), slice(k - 64, k)]
    for part in parts:
        some = part.stop - part.start
        x[:, part] = torch.randint(-4, 5, (2, some), generator=g).float().to(F8).cuda()
        w[0, :, part] = torch.randint(-4, 5, (n, some), generator=g).float().to(F8).cuda()
    xs, ws = torch.ones(2, k // 128, device="cuda"), torch.ones(1, 3, k // 128, device="cuda")
    xs[:, -1] = 2.0
    out = _new(2, n, dtype=torch.bfloat16)
    mlg.mlg_grouped_gemm_f8(x, xs, None, w, ws, out, 2, k, n, 1)
    want = sum(by * (x[:, p].double() @ w[0, :, p].double().t()) for by, p in zip((1, 1, 2), parts))
    assert torch.equal(out, want.to(torch.bfloat16))


@pytest.mark.parametrize("rows", [3, 70])
def test_many_columns(rows):
    n, k, cut = mlg.MLG_F8_MAX_WIDTH, 48, mlg.MLG_F8_MAX_WIDTH - 4096
    w, x, xs = _codes(1, n, k, seed=2), _codes(rows, k, seed=3), torch.ones(rows, 1, device="cuda")
    ws = torch.full((1, n // 128, 1), 0.5, device="cuda")
    out, want = _new(rows, n, dtype=torch.bfloat16), _new(rows, 4096, dtype=torch.bfloat16)
    mlg.mlg_grouped_gemm_f8(x, xs, None, w, ws, out, rows, k, n, 1)
    mlg.mlg_grouped_gemm_f8(x, xs, None, w[:, cut:].contiguous(), ws[:, cut // 128:].contiguous(),
                            want, rows, k, 4096, 1)
    assert torch.equal(out[:, cut:], want)
    ref, err = refs.gemm_f8(*(t.double().cpu().numpy() for t in (x, xs, w[0, :4096], ws[0, :32])))
    operator_refs.assert_within(out[:, :4096].double().cpu().numpy(), ref, err, True)
