"""GPU tests of a plan's first calls on streams that do not wait for the default stream."""
import pytest
import torch

from mixture_experts_layer_19_gb300 import moe
from tests.util import cpu_and_gpu_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ep_ranks,flags", [(0, 0), (0, moe.MOE_DEBUG_RING_MEGAKERNEL), (2, 0)])
def test_a_plan_made_behind_queued_work_is_ready_for_any_stream(ep_ranks, flags):
    T, d, F, E, k = 20, 512, 256, 8, 2
    g, _ = cpu_and_gpu_inputs(T, d, F, E, k, seed=21)
    W = (g["Wg"], g["Wu"], g["Wd"])
    config = moe.Config(T_max=T, d=d, F=F, E=E, k=k, ep_ranks=ep_ranks, debug_flags=flags)
    with moe.Plan(config) as plan:
        few, (Y, _) = plan.forward_few(g["X"], g["logits"], *W), plan.forward(g["X"], g["logits"], *W)
    junk = [torch.full((1 << 22,), 0x7f7f7f7f, dtype=torch.int32, device="cuda") for _ in range(8)]
    busy = torch.randn((8192, 8192), device="cuda")
    side = torch.cuda.Stream()
    del junk
    torch.cuda.empty_cache()                             # a plan's allocations may find these bytes
    torch.cuda.synchronize()
    for _ in range(20):
        busy @ busy
    plan = moe.Plan(config)
    with torch.cuda.stream(side):
        got_few = plan.forward_few(g["X"], g["logits"], *W)
        got_Y, _ = plan.forward(g["X"], g["logits"], *W)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert torch.equal(got_few, few) and torch.equal(got_Y, Y)
    plan.close()
