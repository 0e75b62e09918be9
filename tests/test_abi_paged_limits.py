"""Limits of rra_attend_paged that no GPU is needed for."""
from ragged_attention_token_gb300 import build, rra


def test_units_past_a_grid_go_as_tiles():
    """One CTA a sequence and head is more than a grid may have from 2^31 on: such a call's tiles share a workspace."""
    if not build.up_to_date():
        build.build()
    f = rra.lib().rra_attend_paged_workspace_bytes
    assert f(65535, 1, 1, 3, 32768, 32768, 64) == 0             # 2^31 - 32768 units
    assert f(65535, 1, 1, 3, 32769, 32769, 64) > 0
    assert f(65535, 1, 1, 3, 65535, 65535, 128) > 0
