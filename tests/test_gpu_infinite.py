"""GPU tests of the serving operators where a value between their products is infinite: the formula's infinities come
out, and no other row notices."""
import pytest
import torch

from mixture_experts_layer_19_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.mark.parametrize("T,d,F,E,k", [(1, 256, 256, 2, 2), (5, 512, 1024, 8, 2), (20, 256, 512, 4, 1), (64, 768, 256, 3, 2)])
def test_an_infinite_h_in_the_layer_for_few_tokens(T, d, F, E, k):
    """Positive weights and a token of 2^100: every h overflows, and a column of Y has the sign of its row of Wd."""
    g = torch.Generator(device=DEV).manual_seed(T)
    Wg, Wu = (torch.rand((E, F, d), generator=g, device=DEV).to(BF16) + 0.25 for _ in range(2))
    sign = torch.where(torch.rand(d, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    Wd = ((torch.rand((E, d, F), generator=g, device=DEV) + 0.5) * sign[:, None] / F).to(BF16)
    X = torch.rand((T, d), generator=g, device=DEV).to(BF16)
    logits = torch.randn((T, E), generator=g, device=DEV)
    with moe.Plan(moe.Config(T_max=T, d=d, F=F, E=E, k=k)) as plan:
        ref = plan.forward_few(X, logits, Wg, Wu, Wd)
        assert torch.isfinite(ref).all()
        big = X.clone()
        t = T // 2
        big[t] = 2.0 ** 100
        Y = plan.forward_few(big, logits, Wg, Wu, Wd)
        assert torch.equal(Y[t].float(), sign * float("inf"))
        assert torch.equal(plan.forward(big, logits, Wg, Wu, Wd)[0][t], Y[t])
        keep = [i for i in range(T) if i != t]
        assert torch.equal(Y[keep], ref[keep])
        assert plan.device_status() == 0
