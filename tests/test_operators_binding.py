"""What the binding of the operators around the fold refuses before a call: tensors of another
element type than the call reads, and tensors that are not in the order it reads.  Every refusal
comes before any device work, so this runs without a GPU."""
import sys

import pytest

torch = pytest.importorskip("torch")

import lora_moe_expert_gb300 as mlg  # noqa: E402

T, K, E, W = 4, 2, 8, 64
N = T * K


@pytest.fixture(params=["extension", "ctypes"])
def _through(request, monkeypatch):
    monkeypatch.setattr(mlg, "_native", None)
    if request.param == "ctypes":
        monkeypatch.setitem(sys.modules, "lora_moe_expert_gb300._mlg_py", None)
        monkeypatch.delattr(mlg, "_mlg_py", raising=False)
    else:
        pytest.importorskip("lora_moe_expert_gb300._mlg_py")


def _tensors():
    i32, bf16 = torch.int32, torch.bfloat16
    return dict(
        logits=torch.zeros(T, E), dlogits=torch.zeros(T, E),
        indices=torch.zeros(T, K, dtype=i32), weights=torch.zeros(T, K),
        dweights=torch.zeros(T, K), row_adapter=torch.zeros(T, dtype=i32),
        offsets=torch.zeros(E + 1, dtype=i32), src=torch.zeros(N, dtype=i32),
        pos=torch.zeros(N, dtype=i32), held=torch.zeros(1, dtype=i32),
        x=torch.zeros(T, W, dtype=bf16), rows=torch.zeros(N, W, dtype=bf16),
        out=torch.zeros(T, W, dtype=bf16), codes=torch.zeros(E, 8, W // 2, dtype=torch.uint8),
        scales=torch.zeros(E, 8, 2, dtype=bf16), zeros=torch.zeros(E, 8, 2, dtype=torch.uint8),
        q4_out=torch.zeros(N, 8, dtype=bf16))


# every call, its tensors by name, and those of them with one element type and no stride
CALLS = {
    "route": ((lambda t: mlg.mlg_route_topk(t["logits"], t["indices"], t["weights"], T, E, K, True,
                                            stream=0)), "indices weights"),
    "route_backward": ((lambda t: mlg.mlg_route_topk_backward(
        t["logits"], t["indices"], t["weights"], t["dweights"], t["dlogits"], T, E, K, False,
        stream=0)), "indices weights dweights"),
    "sort": ((lambda t: mlg.mlg_sort_slots(t["indices"], t["row_adapter"], t["offsets"], t["src"],
                                           t["pos"], N, K, E, 1, stream=0)),
             "indices row_adapter offsets src pos"),
    "dispatch": ((lambda t: mlg.mlg_dispatch(
        t["x"], t["indices"], t["row_adapter"], t["offsets"], t["src"], t["pos"], t["rows"], N, W,
        K, E, 1, stream=0)), "indices row_adapter offsets src pos"),
    "combine": ((lambda t: mlg.mlg_combine(t["rows"], t["pos"], t["weights"], t["out"], T, W, K, N,
                                           stream=0)), "pos weights"),
    "combine_backward": ((lambda t: mlg.mlg_combine_backward(
        t["x"], t["rows"], t["pos"], t["weights"], t["held"], t["rows"], t["dweights"], T, W, K, N,
        stream=0)), "pos weights held dweights"),
    "q4": ((lambda t: mlg.mlg_gather_q4(t["x"], t["indices"], t["codes"], t["scales"], t["zeros"],
                                        t["q4_out"], N, W, 8, K, E, 32, stream=0)),
           "x indices codes scales zeros q4_out"),
}
TYPED = [(call, name) for call, (_, names) in CALLS.items() for name in names.split()]


@pytest.mark.parametrize("call,name", TYPED)
def test_other_element_types_are_refused(_through, call, name):
    """int64 ids (what torch.topk gives), fp16 scales, fp32 activations and the like."""
    for dtype in (torch.int64, torch.float16, torch.float32, torch.int32, torch.int8):
        tensors = _tensors()
        if tensors[name].dtype == dtype:
            continue
        tensors[name] = tensors[name].to(dtype)
        with pytest.raises(TypeError):
            CALLS[call][0](tensors)


@pytest.mark.parametrize("call,name", TYPED)
def test_strided_tensors_are_refused(_through, call, name):
    """A slice of wider rows, and one row read as many."""
    tensors = _tensors()
    t = tensors[name]
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
    tensors[name] = wide[..., ::2] if t.dim() == 1 else wide[..., :t.shape[-1]]
    if t.numel() > 1:  # one element has no stride
        with pytest.raises(ValueError):
            CALLS[call][0](tensors)
        tensors[name] = t.reshape(-1)[:1].expand(t.shape)
        with pytest.raises(ValueError):
            CALLS[call][0](tensors)


def test_an_empty_batch_of_the_router_is_a_no_op(_through):
    one = torch.zeros(1, E)
    mlg.mlg_route_topk(one, one, one, 0, E, K, True, stream=0)
    mlg.mlg_route_topk_backward(one, one, one, one, one, 0, E, K, False, stream=0)
    with pytest.raises(mlg.MlgError):
        mlg.mlg_route_topk(one, one, one, 0, 0, K, True, stream=0)


@pytest.mark.parametrize("call,name", [("dispatch", "rows"), ("combine", "rows"),
                                       ("combine_backward", "rows")])
def test_strided_sorted_rows_are_refused(_through, call, name):
    """The token side's rows have a stride of their own; the sorted rows lie one after the other."""
    for rows in (torch.zeros(N, 2 * W, dtype=torch.bfloat16)[:, :W],
                 torch.zeros(1, W, dtype=torch.bfloat16).expand(N, W)):
        tensors = _tensors()
        tensors[name] = rows
        with pytest.raises(ValueError):
            CALLS[call][0](tensors)


@pytest.mark.parametrize("strided", ["y", "dy"])
def test_strided_rows_of_the_gradient_are_refused(_through, strided):
    t = _tensors()
    wide = torch.zeros(N, 2 * W, dtype=torch.bfloat16)[:, :W]
    y, dy = (wide, t["rows"]) if strided == "y" else (t["rows"], wide)
    with pytest.raises(ValueError):
        mlg.mlg_combine_backward(t["x"], y, t["pos"], t["weights"], None, dy, t["dweights"], T, W, K,
                                 N, stream=0)


def test_the_lost_copies_hook_takes_0_and_1():
    for value in (-1, 2):
        with pytest.raises(mlg.MlgError):
            mlg.mlg_test_set_knob(mlg.MLG_TEST_Q4_LOSE, value)
    mlg.mlg_test_set_knob(mlg.MLG_TEST_Q4_LOSE, 0)


def test_addresses_need_their_type_and_stride(_through):
    t, P = _tensors(), 1 << 20
    for type, ld in ((None, None), (None, E), (mlg.MLG_TYPE_F32, None)):
        with pytest.raises(TypeError):
            mlg.mlg_route_topk(P, t["indices"], t["weights"], T, E, K, True, type=type, ld_logits=ld,
                               stream=0)
    mlg.mlg_combine(P, None, None, P, 0, W, K, N, type=mlg.MLG_TYPE_F32, ld_out=W, stream=0)


def test_the_stream_is_asked_for_after_the_checks(_through, monkeypatch):
    asked = []
    monkeypatch.setattr(mlg, "_raw_stream", lambda: asked.append(1) or 0)
    t = _tensors()
    with pytest.raises(TypeError):
        mlg.mlg_route_topk(t["logits"], t["src"].long(), t["weights"], T, E, K, True)
    assert not asked
    mlg.mlg_route_topk(t["logits"], t["indices"], t["weights"], 0, E, K, True)
    assert asked == [1]


def test_rows_of_one_element_have_any_stride(_through):
    one = torch.zeros(T, 2)[:, :1]
    logits = one.as_strided((T, 1), (2, 7))
    mlg.mlg_route_topk(logits, None, None, 0, 1, K, True, stream=0)
    with pytest.raises(ValueError):
        mlg.mlg_route_topk(torch.zeros(E, T).t(), None, None, 0, E, K, True, stream=0)
    with pytest.raises(ValueError):
        mlg.mlg_route_topk(torch.zeros(T * E), None, None, 0, E, K, True, stream=0)
