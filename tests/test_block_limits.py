"""Limits of a whole MoE block's operators that are refused before any device work."""
import pytest

import lora_moe_expert_gb300 as mlg
from test_block_host import CALLS, UNSUPPORTED


def _refused(name, **changes):
    ok = CALLS[name][0]
    assert not set(changes) - set(ok)
    return getattr(mlg.lib(), name)(*{**ok, **changes}.values(), 0) == UNSUPPORTED


def test_a_product_whose_rows_or_columns_leave_32_bits():
    """Counted up to a tile past the last one."""
    for n in (mlg.MLG_F8_MAX_ROWS + 1, (1 << 31) - 1):
        assert _refused("mlg_grouped_gemm_f8", n_rows=n)
    for n in (mlg.MLG_F8_MAX_WIDTH + 16, (1 << 31) - 16):
        assert _refused("mlg_grouped_gemm_f8", k_in=n)
        assert _refused("mlg_grouped_gemm_f8", n_out=n)


def test_weight_gradients_off_their_alignment():
    for name in ("dw_post", "dw_pre"):
        assert _refused("mlg_block_norm_backward", **{name: (1 << 20) + 2})


def test_the_hook_takes_a_truth_value():
    for value in (-1, 2):
        with pytest.raises(mlg.MlgError):
            mlg.mlg_test_set_knob(mlg.MLG_TEST_BLOCK_LOSE, value)
    mlg.mlg_test_set_knob(mlg.MLG_TEST_BLOCK_LOSE, 0)
