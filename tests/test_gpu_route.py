"""The router's top_k weights and their gradient against plain 64-bit forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_refs as refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    yield
    torch.cuda.synchronize()


def _logits(T, E, dtype, seed, kind, pad=0):
    """[T, E] logits as a slice of rows of E + pad, the rest NaN."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((T, E)) * 3
    if kind == "ties":
        v = rng.integers(-2, 3, (T, E)).astype(float)
        v[rng.random((T, E)) < 0.2] = -0.0
    elif kind == "masked":
        v[rng.random((T, E)) < 0.7] = -np.inf
        v[::3] = -np.inf  # rows whose mask leaves nothing
        v[rng.random((T, E)) < 0.05] = np.nan
    elif kind == "lowest":  # masks of the type's lowest value are finite
        v[rng.random((T, E)) < 0.7] = torch.finfo(TYPES[dtype]).min
        v[::4] = torch.finfo(TYPES[dtype]).min
    elif kind == "inf":
        v[rng.random((T, E)) < 0.1] = np.inf
        v[rng.random((T, E)) < 0.3] = -np.inf
    elif kind == "wide":
        v *= 40
    wide = torch.full((T, E + pad), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide[:, :E] = torch.from_numpy(v).to("cuda").to(TYPES[dtype])
    return wide[:, :E], wide


def _run(logits, K, renorm, stream=None):
    T, E = logits.shape
    guard = 16
    idx = torch.full((T * K + guard,), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T * K + guard,), 77.0, device="cuda")
    mlg.mlg_route_topk(logits, idx, w, T, E, K, renorm, stream=stream)
    torch.cuda.synchronize()
    assert (idx[T * K:] == 77).all() and (w[T * K:] == 77).all()
    return idx[:T * K].view(T, K).clone(), w[:T * K].view(T, K).clone()


SHAPES = [(1, 1, 1), (3, 5, 2), (2, 5, 8), (257, 32, 4), (33, 33, 32), (64, 128, 8), (7, 97, 6),
          (65, 256, 8), (19, 511, 10), (40, 512, 10), (9, 513, 1), (12, 1000, 16), (5, 1024, 32)]


@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "lowest", "inf", "wide"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_topk(T, E, K, dtype, kind):
    for renorm, pad in ((True, 0), (False, 3), (False, 8)):
        logits, _ = _logits(T, E, dtype, T * 1000 + E, kind, pad)
        idx, w = _run(logits, K, renorm)
        ref_idx, ref_w, bound = refs.route(logits.float().cpu().numpy(), K, renorm)
        assert np.array_equal(idx.cpu().numpy(), ref_idx)
        refs.assert_within(w.cpu().numpy(), ref_w, bound)
        assert (w.cpu().numpy()[ref_idx < 0] == 0).all()


@pytest.mark.parametrize("kind", ["plain", "masked", "lowest", "wide"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_gradient(T, E, K, dtype, kind):
    rng = np.random.default_rng(E)
    for renorm, pad in ((True, 0), (False, 0), (False, 5), (True, 8), (False, 8)):
        logits, _ = _logits(T, E, dtype, T * 1000 + E, kind, pad)
        idx, w = _run(logits, K, renorm)
        dw = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
        wide = torch.full((T, E + pad), 5.0, dtype=TYPES[dtype], device="cuda")
        mlg.mlg_route_topk_backward(None if renorm else logits, idx, w, dw, wide[:, :E], T, E, K,
                                    renorm)
        ref, bound = refs.route_grad(logits.float().cpu().numpy(), idx.cpu().numpy(),
                                     w.cpu().numpy(), dw.cpu().numpy(), renorm)
        refs.assert_within(wide[:, :E].float().cpu().numpy(), ref,
                           bound, dtype == "bf16")
        assert (wide[:, E:] == 5).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """fp32 gradients against central differences of the 64-bit loss: step 1e-5 leaves ~1e-10 of
    truncation and ~1e-11 of rounding, far below the fp32 error (at most ~1e-5 of O(1) values)."""
    T, E, K, h = 4, 12, 3, 1e-5
    logits, _ = _logits(T, E, "f32", 3, "masked", 0)
    idx, w = _run(logits, K, renorm)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).cuda()
    grad = torch.empty(T, E, device="cuda")
    mlg.mlg_route_topk_backward(logits, idx, w, dw, grad, T, E, K, renorm)
    v, i, d = logits.cpu().double().numpy(), idx.cpu().numpy(), dw.cpu().double().numpy()
    for t in range(T):
        for e in range(E):
            up, down = v.copy(), v.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = (refs.route_loss(up, i, d, renorm) - refs.route_loss(down, i, d, renorm)) / (2 * h)
            assert abs(grad[t, e].item() - diff) < 1e-5, (t, e)


def test_other_stream_graph_and_repeat():
    logits, _ = _logits(300, 200, "bf16", 5, "ties")
    first = _run(logits, 8, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = _run(logits, 8, True, stream=side)
    idx, w = torch.zeros(300, 8, dtype=torch.int32, device="cuda"), torch.zeros(300, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlg.mlg_route_topk(logits, idx, w, 300, 200, 8, True)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in ((again, first), ((idx, w), first)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_tokens():
    one = torch.zeros(1, 8, device="cuda")
    mlg.mlg_route_topk(one, one, one, 0, 8, 2, True)
    mlg.mlg_route_topk_backward(one, one, one, one, one, 0, 8, 2, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,K", [(97, 4), (128, 8), (256, 9), (500, 10), (512, 24), (512, 25), (1024, 32)])
def test_best_experts_together(E, K, dtype):
    """The best 2 to K experts are those of a few residues modulo 64 (or 32), which one lane of the
    warp holds, in any order among the others."""
    rng = np.random.default_rng(E + K)
    T = 96
    v = rng.standard_normal((T, E))
    for t in range(T):
        step = (64, 32)[t % 2]
        first = int(rng.integers(0, step - 1)) & ~1
        ids = np.concatenate([np.arange(first, E, step), np.arange(first + 1, E, step)])
        n = min(2 + t % (K - 1), ids.size)
        v[t, rng.permutation(ids)[:n]] += 4 + 4 * rng.random(n)
    logits = torch.from_numpy(v).cuda().to(TYPES[dtype])
    for renorm in (True, False):
        idx, w = _run(logits, K, renorm)
        ref_idx, ref_w, bound = refs.route(logits.float().cpu().numpy(), K, renorm)
        assert np.array_equal(idx.cpu().numpy(), ref_idx)
        refs.assert_within(w.cpu().numpy(), ref_w, bound)


@pytest.mark.parametrize("E,K", [(128, 4), (200, 8), (512, 10), (1024, 24)])
def test_more_than_three_of_one_lane(E, K):
    """bf16, every token: a lane of the warp holds four or more of the chosen, so that the choices
    are made a second time, mostly by other lanes than the first.  Many warps at once, repeated."""
    rng = np.random.default_rng(E)
    T = 3000
    v = rng.standard_normal((T, E))
    for t in range(T):
        first = 2 * int(rng.integers(0, 32))
        ids = np.concatenate([np.arange(first, E, 64), np.arange(first + 1, E, 64)])
        v[t, ids[rng.permutation(ids.size)[:max(4, K - 1)]]] += 6 + rng.random()
    logits = torch.from_numpy(v).cuda().to(torch.bfloat16)
    ref_idx, ref_w, bound = refs.route(logits.float().cpu().numpy(), K, True)
    for _ in range(5):
        idx, w = _run(logits, K, True)
        assert np.array_equal(idx.cpu().numpy(), ref_idx)
        refs.assert_within(w.cpu().numpy(), ref_w, bound)
