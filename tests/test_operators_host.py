"""Argument checks of the operators around the fold: every refusal comes before any device work,
so this runs without a GPU."""
import pytest

import lora_moe_expert_gb300 as mlg

P = 1 << 20  # a 16-byte-aligned stand-in address; never dereferenced on error paths
INVALID, UNSUPPORTED = mlg.MLG_ERR_INVALID_ARG, mlg.MLG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    return mlg.lib()


def _caller(fn, order, defaults):
    def call(**kw):
        assert not set(kw) - set(order)
        args = {**defaults, **kw}
        return fn(*[args[name] for name in order], 0)

    return call


def test_route_refusals(L):
    order = "logits type ld indices weights n_tokens n_experts top_k renormalize".split()
    ok = dict(logits=P, type=0, ld=16, indices=P, weights=P, n_tokens=4, n_experts=16, top_k=2,
              renormalize=1)
    call = _caller(L.mlg_route_topk, order, ok)
    for bad in (dict(logits=None), dict(indices=None), dict(weights=None), dict(n_tokens=-1),
                dict(n_experts=0), dict(top_k=0), dict(type=2), dict(type=-1), dict(ld=15)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n_experts=1025, ld=1025), dict(top_k=33), dict(logits=P + 1),
                dict(type=1, logits=P + 2)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n_tokens=0) == mlg.MLG_OK

    order = ("logits type ld indices weights dweights dlogits ld_dlogits n_tokens n_experts top_k "
             "renormalize").split()
    ok.update(dweights=P, dlogits=P, ld_dlogits=16)
    call = _caller(L.mlg_route_topk_backward, order, ok)
    for bad in (dict(indices=None), dict(weights=None), dict(dweights=None), dict(dlogits=None),
                dict(renormalize=0, logits=None), dict(renormalize=0, ld=15), dict(ld_dlogits=15),
                dict(n_tokens=-1), dict(n_experts=0), dict(top_k=0), dict(type=7)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n_experts=1025, ld=1025, ld_dlogits=1025), dict(top_k=33),
                dict(dlogits=P + 1), dict(renormalize=0, type=1, logits=P + 2)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n_tokens=0, logits=None) == mlg.MLG_OK


SORT = dict(indices=P, row_adapter=None, offsets=P, src=P, pos=P, n_slots=8, top_k=2, n_experts=4,
            n_adapters=1)
SORT_INVALID = (dict(indices=None), dict(offsets=None), dict(src=None), dict(pos=None),
                dict(n_slots=-1), dict(top_k=0), dict(n_experts=-1), dict(n_adapters=0))
SORT_UNSUPPORTED = (dict(n_experts=mlg.MLG_SORT_MAX_CELLS + 1),
                    dict(n_experts=1024, n_adapters=25, row_adapter=P),
                    dict(n_experts=1 << 30, n_adapters=1 << 30, row_adapter=P))


def test_sort_refusals(L):
    order = "indices row_adapter offsets src pos n_slots top_k n_experts n_adapters".split()
    call = _caller(L.mlg_sort_slots, order, SORT)
    for bad in SORT_INVALID:
        assert call(**bad) == INVALID, bad
    for bad in SORT_UNSUPPORTED:
        assert call(**bad) == UNSUPPORTED, bad


def test_dispatch_refusals(L):
    order = ("x type ld indices row_adapter offsets src pos x_rows n_slots width top_k n_experts "
             "n_adapters").split()
    call = _caller(L.mlg_dispatch, order, {**SORT, "x": P, "type": 0, "ld": 64, "x_rows": P,
                                           "width": 64})
    for bad in SORT_INVALID + (dict(x=None), dict(x_rows=None), dict(width=0), dict(ld=56),
                               dict(type=3)):
        assert call(**bad) == INVALID, bad
    for bad in SORT_UNSUPPORTED + (dict(x=P + 8), dict(x_rows=P + 4), dict(width=60), dict(ld=68),
                                   dict(type=1, width=62), dict(type=1, ld=66)):
        assert call(**bad) == UNSUPPORTED, bad


def test_combine_refusals(L):
    order = "y type pos weights out ld n_tokens width top_k n_rows".split()
    ok = dict(y=P, type=0, pos=P, weights=P, out=P, ld=64, n_tokens=4, width=64, top_k=2, n_rows=8)
    call = _caller(L.mlg_combine, order, ok)
    for bad in (dict(y=None), dict(out=None), dict(n_tokens=-1), dict(width=0), dict(top_k=0),
                dict(n_rows=-1), dict(ld=56), dict(type=2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(y=P + 8), dict(out=P + 2), dict(width=60), dict(ld=68),
                dict(n_tokens=1 << 30, top_k=2)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n_tokens=0) == mlg.MLG_OK

    order = "dout type ld y pos weights held dy dweights n_tokens width top_k n_rows".split()
    ok.update(dout=P, held=None, dy=P, dweights=P)
    call = _caller(L.mlg_combine_backward, order, ok)
    for bad in (dict(dout=None), dict(dy=None), dict(y=None), dict(n_tokens=-1), dict(width=0),
                dict(top_k=0), dict(n_rows=-1), dict(ld=56), dict(type=2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dout=P + 8), dict(dy=P + 8), dict(y=P + 8), dict(width=60), dict(ld=68),
                dict(n_tokens=1 << 30, top_k=2)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n_tokens=0) == mlg.MLG_OK


def test_q4_refusals(L):
    order = "x indices codes scales zeros out n_slots k_in n_out top_k n_experts group".split()
    ok = dict(x=P, indices=P, codes=P, scales=P, zeros=None, out=P, n_slots=8, k_in=128, n_out=64,
              top_k=2, n_experts=4, group=64)
    call = _caller(L.mlg_gather_q4, order, ok)
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(out=None),
                dict(n_slots=-1), dict(k_in=0), dict(n_out=0), dict(top_k=0),
                dict(n_experts=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(group=16), dict(group=0), dict(group=96), dict(k_in=96), dict(n_out=60),
                dict(n_experts=mlg.MLG_Q4_MAX_EXPERTS + 1), dict(x=P + 8), dict(codes=P + 4), dict(out=P + 8), dict(scales=P + 2), dict(zeros=P + 8),
                dict(k_in=64 * (mlg.MLG_Q4_MAX_GROUPS + 1))):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n_slots=0) == mlg.MLG_OK


@pytest.mark.parametrize("ctypes_only", [False, True])
def test_binding_raises_the_status(monkeypatch, ctypes_only):
    """Through the extension module and, where that is not built, through ctypes."""
    import sys

    monkeypatch.setattr(mlg, "_native", None)
    if ctypes_only:
        monkeypatch.setitem(sys.modules, "lora_moe_expert_gb300._mlg_py", None)
        monkeypatch.delattr(mlg, "_mlg_py", raising=False)
    with pytest.raises(mlg.MlgError) as e:
        mlg.mlg_sort_slots(P, None, P, P, P, 8, 0, 4, stream=0)
    assert e.value.status == INVALID
    with pytest.raises(mlg.MlgError) as e:
        mlg.mlg_gather_q4(P, P, P, P, None, P, 8, 128, 64, 2, 4, 16, stream=0)
    assert e.value.status == UNSUPPORTED
    mlg.mlg_combine(P, P, None, P, 0, 64, 2, 8, type=0, ld_out=64, stream=0)


def test_extension_module_checks_its_arguments(L):
    m = pytest.importorskip("lora_moe_expert_gb300._mlg_py")
    with pytest.raises(TypeError):
        m.mlg_sort_slots(P, None, P)
    with pytest.raises(OverflowError):
        m.mlg_sort_slots(P, None, P, P, P, 1 << 40, 1, 4, 1, 0)
    with pytest.raises(AttributeError):
        m.mlg_sort_slots("indices", None, P, P, P, 8, 1, 4, 1, 0)
    with pytest.raises(TypeError):
        m.mlg_sort_slots(P, None, P, P, P, 8.5, 1, 4, 1, 0)


def test_binding_checks_types_and_strides():
    torch = pytest.importorskip("torch")
    bf, f32 = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(TypeError):
        mlg.mlg_route_topk(torch.zeros(4, 64, dtype=torch.float16), i, f32, 4, 64, 2, True)
    with pytest.raises(ValueError):
        mlg.mlg_route_topk(torch.zeros(64, 4).t(), i, f32, 4, 64, 2, True)
    with pytest.raises(TypeError):
        mlg.mlg_dispatch(f32, i, None, i, i, i, bf, 8, 64, 2, 4)
    with pytest.raises(TypeError):
        mlg.mlg_combine(bf, i, None, f32, 4, 64, 2, 8)
    with pytest.raises(TypeError):
        mlg.mlg_combine_backward(bf, f32, i, None, None, bf, f32, 4, 64, 2, 8)
    with pytest.raises(TypeError):
        mlg.mlg_route_topk_backward(bf, i, f32, f32, f32, 4, 64, 2, True)
