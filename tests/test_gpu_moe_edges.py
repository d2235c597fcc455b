"""Calls of the layer that its documentation allows: more choices than experts, calls that run at the
same time on two streams and from two graphs, weights that are not finite."""
import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_moe_layer import Layer  # noqa: E402

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


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 4), (5, 3, 8), (64, 2, 32), (17, 31, 32)])
def test_more_choices_than_experts(T, E, K, f8):
    layer = Layer(T, E, K, 80, 48, f8, T)
    layer.run()
    layer.check()
    assert (layer.indices[:T, E:] == -1).all()


@pytest.mark.parametrize("f8", [False, True])
def test_two_at_the_same_time(f8):
    """Each with workspaces and outputs of its own: on two streams, then as two graphs."""
    layers = [Layer(9, 24, 4, 528, 272, f8, 1), Layer(40, 16, 2, 400, 144, not f8, 2)]
    want = [layer.run().clone() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    graphs = []
    for layer in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.run()
        graphs.append(graph)
    torch.cuda.synchronize()
    for once in ([layer.run for layer in layers], [graph.replay for graph in graphs]):
        for layer in layers:
            layer.out.fill_(77.0)
        torch.cuda.synchronize()
        for _ in range(30):
            for stream, call in zip(streams, once):
                with torch.cuda.stream(stream):
                    call()
        torch.cuda.synchronize()
        for layer, w in zip(layers, want):
            assert torch.equal(layer.out, w)


@pytest.mark.parametrize("f8", [False, True])
def test_a_weight_that_is_not_a_number_stays_in_its_expert(f8):
    """In the gates or ups: the tokens of that expert; in the down rows: one channel of theirs."""
    layer = Layer(20, 6, 2, 144, 80, f8, 3)
    plain = layer.run().clone()
    held = (layer.indices[:20] == 4).any(1)
    assert held.any() and not held.all()
    kept = layer.gate_up.clone()
    layer.gate_up.view(torch.uint8 if f8 else torch.int16)[4, 33, 7] = 0x7f if f8 else 0x7fc0
    out = layer.run()[:20]
    assert out[held].isnan().all() and torch.equal(out[~held], plain[:20][~held])
    layer.gate_up = kept
    layer.down.view(torch.uint8 if f8 else torch.int16)[4, 50, 9] = 0xff if f8 else 0x7fc0
    out = layer.run()[:20]
    assert out[held][:, 50].isnan().all()
    other = torch.arange(144, device="cuda") != 50
    assert torch.equal(out[:, other], plain[:20][:, other])
    assert torch.equal(out[~held], plain[:20][~held])
