"""The scale is checked alike by every call of the image attention (CPU: the calls fail a later check)."""
import pytest

from ragged_attention_token_gb300 import build, rra


@pytest.fixture(scope="module")
def L():
    if not build.up_to_date():
        build.build()
    return rra.lib()


def _attend(L, scale):
    return L.rra_attend(None, 0x2000, 0x3000, 0x4000, 2, 197, 6, 64, scale, rra.RRA_BF16, 0x5000, rra.RRA_BF16, None, 197,
                        None)


def _attend_gather(L, scale):
    return L.rra_attend_gather(None, 0x2000, 0x3000, 0x4000, 0x5000, 2, 197, 6, 64, scale, rra.RRA_BF16, 0x6000,
                               rra.RRA_BF16, None)


@pytest.mark.parametrize("call", [_attend, _attend_gather], ids=["attend", "attend_gather"])
def test_any_finite_scale_is_taken(L, call):
    for scale in (0.0, -0.125, 1e-35, 1e35, 0.125):
        assert call(L, scale) == rra.RRA_ERR_INVALID_ARG and b"is null" in L.rra_last_error_message(), scale
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(L, scale) == rra.RRA_ERR_INVALID_ARG and b"scale" in L.rra_last_error_message(), scale
