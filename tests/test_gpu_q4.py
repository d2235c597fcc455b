"""The 4-bit expert product against a plain 64-bit form."""
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


class Problem:
    def __init__(self, seed, n_slots, top_k, E, k, n, group, zeros, idx):
        rng = np.random.default_rng(seed)
        self.args = (n_slots, k, n, top_k, E, group)
        T = (n_slots + top_k - 1) // top_k
        self.x = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda().to(
            torch.bfloat16)
        self.codes = torch.from_numpy(rng.integers(0, 256, (E, n, k // 2)).astype(np.uint8)).cuda()
        self.scales = torch.from_numpy(
            (rng.random((E, n, k // group)) * 0.2 - 0.05).astype(np.float32)).cuda().to(
                torch.bfloat16)
        self.zeros = (torch.from_numpy(rng.integers(0, 16, (E, n, k // group)).astype(np.uint8))
                      .cuda() if zeros else None)
        self.idx = None if idx is None else torch.from_numpy(
            np.ascontiguousarray(idx, np.int32)).cuda()

    def run(self, stream=None):
        n_slots, _, n = self.args[:3]
        out = torch.full((n_slots + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
        mlg.mlg_gather_q4(self.x, self.idx, self.codes, self.scales, self.zeros, out[1:-1],
                          *self.args, stream=stream)
        torch.cuda.synchronize()
        assert (out[0] == 7).all() and (out[-1] == 7).all()
        return out[1:-1].clone()

    def check(self):
        n_slots, _, _, top_k, E, group = self.args
        ref, err = refs.gather_q4(
            self.x.double().cpu().numpy(), None if self.idx is None else self.idx.cpu().numpy(),
            self.codes.cpu().numpy(), self.scales.double().cpu().numpy(),
            None if self.zeros is None else self.zeros.cpu().numpy(), group, n_slots, top_k)
        out = self.run().double().cpu().numpy()
        refs.assert_within(out, ref, err, True)
        if self.idx is not None:
            i = self.idx.cpu().numpy()
            assert (out[(i < 0) | (i >= E)] == 0).all()


def _ids(seed, n, E, kind):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(n, E - 1)
    if kind == "none":
        return np.where(rng.random(n) < 0.5, -1, E)
    return rng.integers(-1, E + 1, n)


# n_slots, top_k, experts, k, n, group
SHAPES = [(1, 1, 1, 32, 8, 32), (8, 8, 128, 2048, 768, 128), (8, 8, 8, 64, 24, 64),
          (7, 2, 3, 96, 40, 32), (16, 1, 4, 768, 256, 64), (33, 3, 5, 128, 136, 128),
          (64, 8, 16, 384, 72, 128), (130, 10, 9, 160, 264, 32), (300, 4, 7, 640, 88, 128),
          (40, 8, 2, 4096, 104, 64), (512, 8, 128, 256, 48, 32), (3, 1, 2, 8320, 16, 64)]


@pytest.mark.parametrize("kind", ["mixed", "one", "none"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("n_slots,top_k,E,k,n,group", SHAPES)
def test_q4(n_slots, top_k, E, k, n, group, zeros, kind):
    Problem(n_slots + k, n_slots, top_k, E, k, n, group, zeros,
            _ids(n_slots, n_slots, E, kind)).check()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("n_slots,k,group", [(5, 12288, 128), (19, 12288, 32), (2, 24576, 64),
                                             (9, 49152, 128)])
def test_long_k(n_slots, k, group, zeros):
    """k_in whose x rows do not fit beside the rings in shared memory."""
    Problem(k, n_slots, 1, 2, k, 40, group, zeros, _ids(k, n_slots, 2, "mixed")).check()


def test_many_rows_of_few_experts():
    """Jobs by the dozen for one expert, one tile each."""
    Problem(3, 700, 2, 2, 160, 16, 32, True, _ids(9, 700, 2, "mixed")).check()


@pytest.mark.parametrize("n_slots", [1, 5, 8, 9, 17, 32, 33, 100, 257])
def test_dense(n_slots):
    """No indices: every row is expert 0."""
    Problem(n_slots, n_slots, 1, 1, 512, 200, 64, n_slots % 2 == 0, None).check()


def test_exact_integers():
    """Small integers and power-of-two scales: one right answer, bit for bit."""
    rng = np.random.default_rng(0)
    p = Problem(1, 48, 4, 6, 256, 64, 32, True, _ids(5, 48, 6, "mixed"))
    p.x = torch.from_numpy(np.where(rng.random((12, 256)) < 0.03, rng.choice([-1.0, 1.0], (12, 256)),
                                    0.0).astype(np.float32)).cuda().to(torch.bfloat16)
    p.scales = torch.full_like(p.scales, 0.5)
    ref, _ = refs.gather_q4(p.x.double().cpu().numpy(), p.idx.cpu().numpy(),
                            p.codes.cpu().numpy(), p.scales.double().cpu().numpy(),
                            p.zeros.cpu().numpy(), 32, 48, 4)
    assert np.abs(ref).max() < 128 and np.array_equal(p.run().double().cpu().numpy(), ref)


def test_no_experts_and_no_rows():
    out = torch.full((4, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    mlg.mlg_gather_q4(None, idx, None, None, None, out, 4, 32, 16, 1, 0, 32)
    assert (out == 0).all()
    out.fill_(7)
    mlg.mlg_gather_q4(None, None, None, None, None, out, 0, 32, 16, 1, 0, 32)
    assert (out == 7).all()


def test_offsets_past_32_bits():
    """An expert whose codes begin past 2^31 bytes."""
    E, n, k, G = 2800, 768, 2048, 128
    codes = torch.zeros(E, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(E, n, k // G, dtype=torch.bfloat16, device="cuda")
    small = Problem(3, 4, 2, 2, k, n, G, False, np.array([1, 0, 0, 1]))
    codes[[0, E - 1]], scales[[0, E - 1]] = small.codes, small.scales
    want = small.run()
    small.codes, small.scales = codes, scales
    small.idx = torch.tensor([E - 1, 0, 0, E - 1], dtype=torch.int32, device="cuda")
    small.args = (4, k, n, 2, E, G)
    assert torch.equal(small.run(), want)


def test_other_stream_graph_and_repeat():
    p = Problem(2, 77, 7, 12, 512, 136, 64, True, _ids(3, 77, 12, "mixed"))
    first = p.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(p.run(stream=side), first)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlg.mlg_gather_q4(p.x, p.idx, p.codes, p.scales, p.zeros, out, *p.args)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("k,group", [(256, 128), (96, 32), (12288, 64)])
def test_nonfinite_inputs_stay_in_their_rows(k, group):
    """Tokens of NaN and infinities beside finite ones; dropped rows of them are zeros."""
    p = Problem(4, 60, 3, 4, k, 40, group, True, _ids(6, 60, 4, "mixed"))
    want = p.run()
    bad = torch.tensor([2, 7, 19])
    p.x[bad[0]], p.x[bad[1], 5], p.x[bad[2]] = float("nan"), float("inf"), float("-inf")
    got, i = p.run(), p.idx.cpu().numpy()
    hit = np.isin(np.arange(60) // 3, bad.numpy()) & (i >= 0) & (i < 4)
    assert torch.equal(got[~torch.from_numpy(hit).cuda()], want[~torch.from_numpy(hit).cuda()])
    assert not torch.isfinite(got[torch.from_numpy(hit & (np.arange(60) // 3 != 7)).cuda()]).any()
