"""GPU test of what a plan holds for the layer for few tokens: parts of cut tiles for as many tokens as its calls have."""
import pytest
import torch

from mixture_experts_layer_19_gb300 import moe

pytestmark = pytest.mark.gpu


def bytes_of(**kw):
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    with moe.Plan(moe.Config(d=256, F=256, E=4, k=1, **kw)):
        return before - torch.cuda.mem_get_info()[0]


def test_plans_hold_as_much_as_their_calls_need():
    bytes_of(T_max=1)                                    # what only a first plan allocates
    one, most, identity = bytes_of(T_max=1), bytes_of(T_max=64), bytes_of(T_max=64, debug_flags=moe.MOE_DEBUG_IDENTITY_EXPERTS)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    parts = 4 * sms * 63 * 1024                          # of 64 tokens, but for one
    assert most - one > 0.9 * parts and most - identity > 0.9 * parts, (one, most, identity)
