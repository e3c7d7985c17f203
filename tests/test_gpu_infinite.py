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


@pytest.mark.parametrize("T,d,n,r", [(1, 512, 3, 8), (40, 512, 3, 24), (300, 512, 3, 40),        # u by dot products
                                     (600, 2048, 2, 64), (1100, 2048, 9, 64)])                   # and by products of tiles
def test_an_infinite_low_side_of_a_projection(T, d, n, r):
    """Positive A and a token of 2^127: every u overflows, and a column of the result has the sign of its row of B.  A
    second token whose u is finite, but past the largest bf16 value."""
    from mixture_experts_layer_19_gb300 import serve, train
    N = 300
    g = torch.Generator(device=DEV).manual_seed(T)
    A = (torch.rand((n, r, d), generator=g, device=DEV) + 0.5).to(BF16)
    sign = torch.where(torch.rand(N, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    B = ((torch.rand((n, N, r), generator=g, device=DEV) + 0.5) * sign[:, None] * 2.0 ** -20).to(BF16)
    W = torch.rand((N, d), generator=g, device=DEV).to(BF16) * 2.0 ** -20
    X = torch.rand((T, d), generator=g, device=DEV).to(BF16)
    ids = torch.arange(T, device=DEV) % n
    ids[T // 2] = ids[T // 3] = 0
    for out in (torch.float32, BF16):
        ref = serve.linear(X, W, A, B, ids, out_dtype=out)
        big = X.clone()
        big[T // 2] = 2.0 ** 127
        got = serve.linear(big, W, A, B, ids, out_dtype=out)
        assert torch.equal(got[T // 2].float(), sign * float("inf"))
        keep = [i for i in range(T) if i != T // 2]
        assert torch.equal(got[keep], ref[keep])
    big = X.clone()
    big[T // 3] = 0
    big[T // 3, 0], big[T // 3, 1] = torch.finfo(BF16).max, 1e36
    A[0, :, :2] = 1.0
    u = big[T // 3, :2].double().sum()                       # the same for every rank index
    assert torch.finfo(BF16).max * (1 + 2.0 ** -9) < u < torch.finfo(torch.float32).max
    got = serve.linear(big, W, A, B, ids, out_dtype=torch.float32)
    exact = big[T // 3].double() @ W.double().T + u * B[0].double().sum(1)
    # r products of three parts and one of W, each addition off by 2^-23 of magnitudes that r u |B| and |x| |W| bound
    size = big[T // 3].double().abs() @ W.double().abs().T + u * B[0].double().abs().sum(1)
    assert ((got[T // 3].double() - exact).abs() <= 2.0 ** -16 * size).all()
    assert train.device_status(0) == 0
