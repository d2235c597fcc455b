"""Rows into expert order and back, and the gradients, against plain 64-bit forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_refs as refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 16
U_PRODUCT = refs.U  # weight * dout is one fp32 product


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    yield
    torch.cuda.synchronize()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _rows(rng, n, width, dtype, pad=0):
    """[n, width] rows inside rows of width + pad, values of the type."""
    v = torch.from_numpy(rng.standard_normal((n, width + pad)).astype(np.float32)).cuda()
    return v.to(TYPES[dtype])[:, :width]


def _f64(t):
    return t.double().cpu().numpy()


def _sort(indices, row_adapter, top_k, E, A, stream=None):
    n = indices.size
    cells = E * (A if row_adapter is not None else 1)
    out = [torch.full((k + GUARD,), -77, dtype=torch.int32, device="cuda")
           for k in (cells + 1, n, n)]
    mlg.mlg_sort_slots(_i32(indices), None if row_adapter is None else _i32(row_adapter), *out, n,
                       top_k, E, A, stream=stream)
    torch.cuda.synchronize()
    got = []
    for t, k in zip(out, (cells + 1, n, n)):
        assert (t[k:] == -77).all()
        got.append(t[:k].cpu().numpy())
    return got


def _ids(rng, n, E, kind):
    if kind == "one":
        return np.full(n, E - 1)
    if kind == "none":
        return np.where(rng.random(n) < 0.5, -1, E)
    if kind == "skewed":
        return np.minimum((rng.random(n) ** 4 * E).astype(np.int64), E - 1)
    return rng.integers(-1, E + 1, n)  # some out of range on both sides


@pytest.mark.parametrize("kind", ["mixed", "skewed", "one", "none"])
@pytest.mark.parametrize("n,top_k,E,A", [
    (1, 1, 1, 0), (7, 2, 3, 0), (33, 8, 5, 2), (512, 8, 128, 0), (513, 8, 128, 1),
    (2048, 8, 128, 4), (2049, 10, 97, 3), (5000, 7, 512, 0), (8191, 3, 2048, 4), (32768, 8, 128, 0),
    (40001, 6, 60, 5), (163840, 10, 512, 0), (300007, 9, 511, 4), (4000, 4, 24576, 0),
    (1025, 1, 0, 0)])
def test_sort(n, top_k, E, A, kind):
    rng = np.random.default_rng(n + E)
    idx = _ids(rng, n, E, kind) if E else np.zeros(n, np.int64)
    ra = rng.integers(-1, A + 1, (n + top_k - 1) // top_k) if A else None
    got = _sort(idx, ra, top_k, E, max(A, 1))
    for g, r, name in zip(got, refs.sort_slots(idx, ra, top_k, E, A), ("offsets", "src", "pos")):
        assert np.array_equal(g, r), name


def test_sort_nothing():
    offsets, _, _ = _sort(np.zeros(0), None, 4, 9, 1)
    assert (offsets == 0).all()


def _dispatch(x, idx, ra, top_k, E, A, width, dtype, stream=None):
    n = idx.size
    cells = E * (A if ra is not None else 1)
    off, src, pos = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (cells + 1, n, n))
    rows = torch.full((n + 2, width), 7.0, dtype=TYPES[dtype], device="cuda")
    mlg.mlg_dispatch(x, _i32(idx), None if ra is None else _i32(ra), off, src, pos, rows[1:-1], n,
                     width, top_k, E, A, stream=stream)
    torch.cuda.synchronize()
    assert (rows[0] == 7).all() and (rows[-1] == 7).all()
    return off.cpu().numpy(), src.cpu().numpy(), pos.cpu().numpy(), rows[1:-1].clone()


DISPATCH = [(1, 1, 1, 0, 8), (1, 8, 128, 0, 2048), (8, 2, 4, 2, 64), (17, 3, 5, 0, 1000),
            (64, 8, 128, 0, 2048), (65, 8, 128, 2, 768), (255, 10, 512, 0, 136),
            (300, 7, 96, 4, 4104), (5000, 2, 60, 0, 72), (700, 10, 512, 3, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,A,width", DISPATCH)
def test_dispatch(T, K, E, A, width, dtype):
    rng = np.random.default_rng(T + width)
    for ragged in (0, K - 1):
        n = T * K - ragged  # the last token may have fewer slots
        idx = _ids(rng, n, E, "mixed")
        ra = rng.integers(-1, A, T) if A else None
        x = _rows(rng, T, width, dtype, pad=8 if ragged else 0)
        got = _dispatch(x, idx, ra, K, E, max(A, 1), width, dtype)
        ref = refs.sort_slots(idx, ra, K, E, A)
        for g, r in zip(got, ref):
            assert np.array_equal(g, r)
        want = _f64(x)[ref[1] // K]
        want[ref[0][-1]:] = 0
        assert np.array_equal(_f64(got[3]), want)


def test_dispatch_keeps_bits():
    """NaN payloads, infinities and -0 are copied as they are."""
    bits = torch.randint(0, 1 << 16, (9, 64), dtype=torch.int32, device="cuda").to(torch.int16)
    idx = np.arange(18) % 4
    got = _dispatch(bits.view(torch.bfloat16), idx, None, 2, 4, 1, 64, "bf16")
    src = torch.from_numpy(got[1].astype(np.int64)).cuda()
    assert torch.equal(got[3].view(torch.int16), bits[src // 2])


ROWS = [(1, 1, 8), (1, 8, 2048), (3, 2, 64), (64, 8, 2048), (65, 7, 1000), (130, 10, 136),
        (33, 32, 520), (9, 33, 264), (1000, 4, 72), (40, 6, 8200)]


def _routed(rng, T, K, E=16):
    idx = _ids(rng, T * K, E, "mixed")
    off, _, pos = refs.sort_slots(idx, None, K, E, 0)
    return int(off[-1]), pos


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,width", ROWS)
def test_combine(T, K, width, dtype):
    rng = np.random.default_rng(T * K)
    n = T * K
    held, pos = _routed(rng, T, K)
    y = _rows(rng, n, width, dtype).contiguous()
    y[held:] = float("nan")  # rows nobody names
    w = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
    for weights, pad in ((w, 0), (None, 8), (w, 8)):
        wide = torch.full((T + 1, width + pad), 7.0, dtype=TYPES[dtype], device="cuda")
        out = wide[:T, :width]
        mlg.mlg_combine(y, _i32(pos), weights, out, T, width, K, n)
        ref, err = refs.combine(_f64(y), pos, None if weights is None else _f64(w), T, K)
        refs.assert_within(_f64(out), ref, err, dtype == "bf16")
        assert (wide[T] == 7).all() and (wide[:, width:] == 7).all()
        assert (_f64(out)[(pos.reshape(T, K) < 0).all(1)] == 0).all()
    # flat order (decode), and positions at or past n_rows contribute nothing
    y = _rows(rng, n, width, dtype).contiguous()
    out = torch.empty(T, width, dtype=TYPES[dtype], device="cuda")
    mlg.mlg_combine(y, None, w, out, T, width, K, n)
    ref, err = refs.combine(_f64(y), np.arange(n), _f64(w), T, K)
    refs.assert_within(_f64(out), ref, err, dtype == "bf16")
    few = max(n // 2, 1)
    mlg.mlg_combine(y, _i32(pos), w, out, T, width, K, few)
    ref, err = refs.combine(_f64(y)[:few], pos, _f64(w), T, K)
    refs.assert_within(_f64(out), ref, err, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,width", ROWS)
def test_combine_gradient(T, K, width, dtype):
    rng = np.random.default_rng(T * K + 1)
    n = T * K
    held, pos = _routed(rng, T, K)
    y = _rows(rng, n, width, dtype).contiguous()
    y[held:] = float("nan")
    w = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
    rows_held = _i32([held])
    for flat, weights, zero_rest, want_dw, pad in ((False, w, True, True, 8),
                                                   (False, w, False, True, 0),
                                                   (False, None, True, True, 0),
                                                   (False, w, True, False, 0),
                                                   (True, w, False, True, 0)):
        at = np.arange(n) if flat else pos
        if flat:
            y = _rows(rng, n, width, dtype).contiguous()
        d = _rows(rng, T, width, dtype, pad)
        dy = torch.full((n + 1, width), 7.0, dtype=TYPES[dtype], device="cuda")
        dw = torch.full((n + GUARD,), 7.0, device="cuda")
        mlg.mlg_combine_backward(d, y if want_dw else None, None if flat else _i32(pos), weights,
                                 rows_held if zero_rest else None, dy, dw if want_dw else None, T,
                                 width, K, n)
        ref, named, ref_dw, err = refs.combine_grad(
            _f64(d), np.nan_to_num(_f64(y)), at, None if weights is None else _f64(w), n, K)
        got = _f64(dy)
        refs.assert_within(got[:n][named], ref[named],
                           U_PRODUCT * np.abs(ref[named]), dtype == "bf16")
        assert (got[:n][~named] == (0.0 if zero_rest else 7.0)).all() and (got[n] == 7).all()
        if want_dw:
            refs.assert_within(_f64(dw)[:n].reshape(T, K), ref_dw, err, False)
            assert (dw[n:] == 7).all()
        else:
            assert (dw == 7).all()


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit sum: the loss is bilinear,
    so a step of 1e-3 is exact up to ~1e-12 and what is left is the kernels' fp32 error."""
    T, K, width, h = 5, 3, 24, 1e-3
    rng = np.random.default_rng(0)
    held, pos = _routed(rng, T, K, 4)
    n = T * K
    y, d = _rows(rng, n, width, "f32"), _rows(rng, T, width, "f32")
    w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    dy, dw = torch.empty(n, width, device="cuda"), torch.empty(T, K, device="cuda")
    mlg.mlg_combine_backward(d, y, _i32(pos), w, _i32([held]), dy, dw, T, width, K, n)

    def loss(yy, ww):
        return float((refs.combine(yy, pos, ww, T, K)[0] * _f64(d)).sum())

    for _ in range(20):
        vy, vw = rng.standard_normal((n, width)), rng.standard_normal((T, K))
        num = (loss(_f64(y) + h * vy, _f64(w)) - loss(_f64(y) - h * vy, _f64(w))) / (2 * h)
        assert abs(num - float((_f64(dy) * vy).sum())) < 1e-4
        num = (loss(_f64(y), _f64(w) + h * vw) - loss(_f64(y), _f64(w) - h * vw)) / (2 * h)
        assert abs(num - float((_f64(dw) * vw).sum())) < 1e-4


def test_dispatch_gradient_is_the_unweighted_combine():
    """<dispatch(x), g> == <x, combine(g)>, shared rows (a token's top_k copies) summed."""
    rng = np.random.default_rng(2)
    T, K, E, width = 37, 5, 6, 40
    idx = _ids(rng, T * K, E, "mixed")
    x, g = _rows(rng, T, width, "f32"), _rows(rng, T * K, width, "f32")
    _, _, pos, rows = _dispatch(x, idx, None, K, E, 1, width, "f32")
    dx = torch.empty(T, width, device="cuda")
    mlg.mlg_combine(g, _i32(pos), None, dx, T, width, K, T * K)
    assert abs(float((_f64(rows) * _f64(g)).sum()) - float((_f64(x) * _f64(dx)).sum())) < 1e-3


def test_offsets_past_32_bits():
    """Rows past 2^32 bytes (and 2^31 elements) of a row buffer."""
    width, n = 2048, 1_200_000
    y = torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")
    far = np.array([0, n - 1, 1_048_576, 1_100_001, n - 2, 524_288])
    vals = _rows(np.random.default_rng(0), far.size, width, "bf16")
    y[torch.from_numpy(far).cuda()] = vals
    w = torch.full((3, 2), 0.5, device="cuda")
    out = torch.empty(3, width, dtype=torch.bfloat16, device="cuda")
    mlg.mlg_combine(y, _i32(far), w, out, 3, width, 2, n)
    ref = _f64(vals).reshape(3, 2, width).sum(1) / 2
    refs.assert_within(_f64(out), ref, refs.sum_bound(2, np.abs(ref) + 8), True)
    dw = torch.empty(3, 2, device="cuda")
    dy = torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")
    mlg.mlg_combine_backward(out, y, _i32(far), w, None, dy, dw, 3, width, 2, n)
    got = dy[torch.from_numpy(far).cuda()]
    assert torch.equal(got.float(), (out.float() * 0.5).repeat_interleave(2, 0))
    assert int(dy.any(1).sum()) == far.size


def test_side_stream_graph_and_repeat():
    rng = np.random.default_rng(4)
    T, K, E, width = 333, 8, 64, 512
    idx = _ids(rng, T * K, E, "mixed")
    x = _rows(rng, T, width, "bf16")
    first = _dispatch(x, idx, None, K, E, 1, width, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = _dispatch(x, idx, None, K, E, 1, width, "bf16", stream=side)
    assert all(np.array_equal(a, b) for a, b in zip(again[:3], first[:3]))
    assert torch.equal(again[3], first[3])
    n = T * K
    ids = _i32(idx)
    off, src, pos = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (E + 1, n, n))
    rows = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(T, K, device="cuda")
    dy, dw = torch.empty_like(rows), torch.empty(T, K, device="cuda")

    def chain():
        mlg.mlg_dispatch(x, ids, None, off, src, pos, rows, n, width, K, E)
        mlg.mlg_combine(rows, pos, w, out, T, width, K, n)
        mlg.mlg_combine_backward(out, rows, pos, w, off[-1:], dy, dw, T, width, K, n)
        return [t.clone() for t in (off, src, pos, rows, out, dy, dw)]

    one, two = chain(), chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three = chain()
    for t in three:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(one, two, three):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("held", [0, 2])
def test_gradient_without_tokens_zeroes_the_rows(held):
    dy = torch.full((5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dout = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    mlg.mlg_combine_backward(dout, None, None, None, _i32([held]), dy, None, 0, 64, 2, 4)
    torch.cuda.synchronize()
    assert (dy[held:4] == 0).all() and (dy[:held] == 7).all() and (dy[4] == 7).all()
    dy.fill_(7)
    mlg.mlg_combine_backward(dout, None, None, None, None, dy, None, 0, 64, 2, 4)
    torch.cuda.synchronize()
    assert (dy == 7).all()


def test_dispatch_sees_what_the_kernel_before_wrote():
    """x and the ids are written right before each dispatch, by kernels of the same stream."""
    T, K, E, width = 3000, 3, 40, 256
    rng = np.random.default_rng(8)
    xs = [_rows(rng, T, width, "bf16") for _ in range(6)]
    ids = [_i32(rng.integers(0, E, T * K)) for _ in range(6)]
    x, idx = torch.zeros_like(xs[0]), torch.zeros_like(ids[0])
    off, src, pos = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (E + 1, T * K, T * K))
    rows = [torch.empty(T * K, width, dtype=torch.bfloat16, device="cuda") for _ in range(24)]
    for i, r in enumerate(rows):
        torch.add(ids[i % 6], 0, out=idx)
        torch.mul(xs[i % 6], 1.0, out=x)
        mlg.mlg_dispatch(x, idx, None, off, src, pos, r, T * K, width, K, E)
    torch.cuda.synchronize()
    for i, r in enumerate(rows):
        order = torch.argsort(ids[i % 6].long(), stable=True)
        assert torch.equal(r, xs[i % 6][order // K]), i


@pytest.mark.parametrize("T,K,E,A,width", [(60, 10, 96, 0, 64), (100, 10, 512, 2, 72), (20, 32, 40, 0, 264),
                                           (3, 41, 7, 3, 8), (600, 1, 33, 0, 136), (724, 1, 4096, 0, 16),
                                           (1500, 1, 33, 2, 64), (510, 2, 60, 1, 80)])
def test_dispatch_few_and_many_slots_a_token(T, K, E, A, width):
    test_dispatch(T, K, E, A, width, "bf16")


@pytest.mark.parametrize("kind", ["mixed", "one"])
@pytest.mark.parametrize("n,top_k,E,A", [(163840, 8, 512, 48), (50001, 3, 8192, 0),
                                         (131072, 8, 1024, 5), (40000, 1, 24575, 0)])
def test_sort_of_many_cells_and_many_slots(n, top_k, E, A, kind):
    """Few warps have room for a histogram: each walks its slots in many steps."""
    test_sort(n, top_k, E, A, kind)
