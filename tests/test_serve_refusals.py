"""Refusals of the serving operators that need no GPU."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_19_gb300 import build as b
    b.build()
    from mixture_experts_layer_19_gb300 import moe
    return moe.load_library()


def test_given_weight_scales_need_a_plan(lib):
    assert lib.moe_quantize_weights_scaled(None, *[None] * 5) == 1
    assert b"null plan" in lib.moe_last_error()
