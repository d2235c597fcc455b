"""The operators together: a MoE projection's prefill, decode and router gradient against plain
64-bit forms.

Tolerances, from the roundings on the way: a row is rounded to bf16 (2^-8 relative at most; twice in
decode, after the product and after the fold), weighted with weights that sum to 1, and the sum is
rounded once more.  Everything else is fp32.  So an output is within (roundings) * 2^-8 of
sum_k w_k |y_k|, and a dweight within 2^-8 of sum |dout y| plus fp32's part."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_refs as refs  # noqa: E402
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


def _f64(t):
    return t.double().cpu().numpy()


def _experts_rows(p, x, indices, w, folds):
    """y [tokens, top_k, n_out] of every slot, unrounded, and of which slots; w [E, n, k]."""
    T, K = indices.shape
    y = np.zeros((T, K, p.n_out))
    pairs = {e: i for i, e in enumerate(range(0, p.n_experts, 2))}
    A, B, scale = _f64(p.A), _f64(p.B), p.scale_table.cpu().numpy()
    for t in range(T):
        for j, e in enumerate(indices[t]):
            if e < 0:
                continue
            y[t, j] = w[e] @ x[t]
            if e in pairs and folds[t]:
                y[t, j] += scale[e] * (B[pairs[e]] @ (A[pairs[e]] @ x[t]))
    return y


def _batch(p, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, p.k_in, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, p.n_experts, generator=g, device="cuda").to(torch.bfloat16)
    logits[T // 2] = -float("inf")  # a padding row: no expert
    logits[0, 3:] = -float("inf")   # fewer experts than top_k
    return x, logits


@pytest.mark.parametrize("T,seed", [(1, 0), (7, 1), (33, 2)])
def test_prefill_and_gradient(T, seed):
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(seed, 10, 96, 72, 4, 16, 32)
    x, logits = _batch(p, T, seed)
    out = p.prefill(x, logits)
    idx, w, _ = refs.route(logits.float().cpu().numpy(), p.top_k, True)
    y = _experts_rows(p, _f64(x), idx, _f64(p.w), np.ones(T, bool))
    ref = (w[:, :, None] * y).sum(1)
    mag = (w[:, :, None] * np.abs(y)).sum(1)
    assert (np.abs(_f64(out) - ref) <= 2 * 2.0 ** -8 * mag + 1e-4 * mag.max()).all()
    assert (_f64(out)[(idx < 0).all(1)] == 0).all()

    dout = torch.randn(T, p.n_out, device="cuda").to(torch.bfloat16)
    dy_rows, dlogits = p.backward(dout)
    d = _f64(dout)
    dw = (d[:, None, :] * y).sum(2)
    dw_mag = (np.abs(d[:, None, :]) * np.abs(y)).sum(2)
    grad, _ = refs.route_grad(logits.float().cpu().numpy(), idx, w, dw, True)
    # the weights' gradient carries the rows' rounding into every chosen logit, then one rounding
    err = 2 * 2.0 ** -8 * (w * dw_mag).sum(1, keepdims=True) + 2.0 ** -8 * np.abs(grad) + 1e-5
    assert (np.abs(_f64(dlogits) - grad) <= err).all()
    assert (_f64(dlogits)[(idx < 0).all(1)] == 0).all()
    # <dy, y> over the rows is <dout, out> (both sides' roundings: 2^-8 of sum |dout| w |y| each)
    pos = p.saved[4].cpu().numpy().reshape(T, p.top_k)
    for t in range(T):
        for j in range(p.top_k):
            if idx[t, j] >= 0:
                want = w[t, j] * d[t]
                assert (np.abs(_f64(dy_rows[pos[t, j]]) - want)
                        <= (2.0 ** -8 + 1e-5) * np.abs(want) + 1e-30).all()
    assert (_f64(dy_rows)[int((idx >= 0).sum()):] == 0).all()
    dx_rows = torch.randn(T * p.top_k, p.k_in, device="cuda").to(torch.bfloat16)
    dx = _f64(p.rows_backward(dx_rows))
    ref_dx, err = refs.combine(_f64(dx_rows), pos, None, T, p.top_k)
    refs.assert_within(dx, ref_dx, err, True)


@pytest.mark.parametrize("T,seed", [(1, 0), (7, 1), (33, 2)])
def test_decode(T, seed):
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(seed, 10, 96, 72, 4, 16, 32)
    x, logits = _batch(p, T, seed)
    row_map = torch.tensor([t % 3 - 1 for t in range(T)], dtype=torch.int32, device="cuda")
    out = p.decode(x, logits, row_map)
    idx, w, _ = refs.route(logits.float().cpu().numpy(), p.top_k, True)
    codes, scales, zeros, group = p.q4
    dense = refs.q4_weights(codes.cpu().numpy(), _f64(scales), zeros.cpu().numpy(), group)
    folds = row_map.cpu().numpy() >= 0
    y = _experts_rows(p, _f64(x), idx, dense, folds)
    base = _experts_rows(p, _f64(x), idx, dense, np.zeros(T, bool))
    ref = (w[:, :, None] * y).sum(1)
    mag = (w[:, :, None] * (np.abs(y) + np.abs(base))).sum(1)
    assert (np.abs(_f64(out) - ref) <= 2 * 2.0 ** -8 * mag + 1e-4 * mag.max()).all()
    assert (_f64(out)[(idx < 0).all(1)] == 0).all()


def test_captured_in_a_graph():
    """Every call reads its routing on the device: a replay with other logits is another batch."""
    from lora_moe_expert_gb300.projection import random_projection

    p = random_projection(4, 16, 128, 64, 2, 16, 64)
    x, logits = _batch(p, 40, 5)
    row_map = torch.zeros(40, dtype=torch.int32, device="cuda")
    other = logits.flip(0).contiguous()
    want = (p.prefill(x, other).clone(), p.decode(x, other, row_map).clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = p.prefill(x, logits), p.decode(x, logits, row_map)
    logits.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
