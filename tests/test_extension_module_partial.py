"""The extension module with a library that lacks calls (an older one beside it): they are refused by
name, and the others work."""
import pytest

from test_extension_module import module  # noqa: F401  (its stand-in has none of a block's calls)

MISSING = ("mlg_rows_f8", "mlg_swiglu_f8", "mlg_grouped_gemm_f8", "mlg_moe_layer", "mlg_moe_layer_f8",
           "mlg_block_norm", "mlg_block_norm_backward")


@pytest.mark.parametrize("name", MISSING)
def test_a_call_that_is_not_there_is_refused(module, name):  # noqa: F811
    with pytest.raises(NotImplementedError, match=name):
        getattr(module, name)(*[0] * 10)
    with pytest.raises(NotImplementedError, match=name):
        getattr(module, name)()


def test_the_others_work(module):  # noqa: F811
    assert module.mlg_sort_slots(0, None, 0, 0, 0, 8, 1, 4, 1, 0) == 0
    with pytest.raises(TypeError, match="10 arguments"):
        module.mlg_sort_slots(0)
