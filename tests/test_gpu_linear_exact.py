"""GPU tests of fp32 results of the projection in norm (tests/linear_norm.py has the bound, and tests/test_linear_norm.py
what it tells apart), and of weights that really pass 2^32 bytes."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300.workload import to_f64
from tests import linear_norm
from tests.test_gpu_linear import CASES, check, inputs, on

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def serve():
    from mixture_experts_layer_19_gb300 import serve, train
    yield serve
    assert train.device_status(0) == 0


def exact(s):
    ref = to_f64(s["X"]) @ to_f64(s["W"]).T
    if "A" in s:
        X, A, B, ids = to_f64(s["X"]), to_f64(s["A"]), to_f64(s["B"]), s["adapter_ids"].numpy()
        for a in range(A.shape[0]):
            t = np.nonzero(ids == a)[0]
            ref[t] += (float(s["scale"][a]) if "scale" in s else 1.0) * (X[t] @ A[a].T) @ B[a].T
    return ref


@pytest.mark.parametrize("T,d,N,n,r", [c for c in CASES if c[0] * c[2] >= 100] + [   # the bound is a norm's: of many values
    (1, 7168, 3000, 0, 8), (64, 8192, 2000, 0, 8), (50, 4096, 5000, 6, 16), (100, 8192, 700, 0, 8), (900, 4096, 1000, 5, 16)])
def test_fp32_results_in_norm(serve, T, d, N, n, r):
    s = inputs(T, d, N, n, r, scale=T % 2 == 0, seed=T + d)
    got = serve.linear(**on(s), out_dtype=torch.float32)
    assert linear_norm.off(to_f64(got), exact(s)) <= linear_norm.tolerance(r if n else 0)


@pytest.mark.parametrize("T,d,N,n,r", [
    (1, 2048, 900, 1, 64), (7, 512, 1001, 2, 8), (40, 2048, 640, 3, 24), (64, 1024, 300, 5, 64),       # up to 64 tokens
    (100, 512, 640, 3, 16), (300, 2048, 640, 4, 40), (128, 1024, 257, 2, 64),                          # u by dot products
    (600, 2048, 640, 2, 64), (1100, 2048, 640, 9, 64), (4000, 2048, 200, 5, 16)])                      # and by products
def test_adapters_that_outweigh_w_in_norm(serve, T, d, N, n, r):
    """W is 2^-12 of the adapters' part, so the third part of u shows."""
    s = inputs(T, d, N, n, r, ids=torch.arange(T) % n, scale=False, seed=T)
    s["W"] = (s["W"].float() * 2.0 ** -12).to(torch.bfloat16)
    got = serve.linear(**on(s), out_dtype=torch.float32)
    assert linear_norm.off(to_f64(got), exact(s)) <= linear_norm.tolerance(r)


@pytest.mark.parametrize("T,out", [(40, torch.float32), (200, torch.bfloat16), (130, torch.float32)])
def test_weights_past_32_bits(serve, T, out):
    """W of 2^33 bytes and more, for up to 64 tokens, on pairs of CTAs and on single ones; the rows at its two ends and where
    it passes 2^32 bytes are not zero."""
    d, n, r, N = 512, 2, 8, (1 << 23) + 300
    g = torch.Generator(device=DEV).manual_seed(T)
    W = torch.zeros((N, d), dtype=torch.bfloat16, device=DEV)
    B = torch.zeros((n, N, r), dtype=torch.bfloat16, device=DEV)
    middle = (1 << 32) // (2 * d)
    parts = [slice(0, 300), slice(middle - 150, middle + 150), slice(N - 300, N)]
    for p in parts:
        W[p] = (torch.randn((300, d), generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
        B[:, p] = torch.randn((n, 300, r), generator=g, device=DEV).to(torch.bfloat16)
    A = (torch.randn((n, r, d), generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    X = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.arange(T, device=DEV) % (n + 1)
    got = serve.linear(X, W, A, B, ids, out_dtype=out)
    for p in parts:
        s = {"X": X, "W": W[p], "A": A, "B": B[:, p], "adapter_ids": ids}
        check(got[:, p].cpu(), {k: v.cpu() for k, v in s.items()})
    for a, b in zip(parts, parts[1:]):
        assert not bool(got[:, a.stop:b.start].any())
