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


def test_sampling_logits_take_no_stream():
    """Only the second of its two calls could run there, beside the first, whose result it needs."""
    from mixture_experts_layer_19_gb300 import train

    class Head:
        def logits(self, *args):
            raise AssertionError("work was enqueued")
    for stream in (None, object()):
        with pytest.raises(ValueError, match="stream"):
            train.LMHead.sampling_logits(Head(), None, stream=stream)
