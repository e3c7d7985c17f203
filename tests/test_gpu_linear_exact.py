"""GPU tests of fp32 results of the projection in norm (tests/linear_norm.py has the bound, and tests/test_linear_norm.py
what it tells apart)."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300.workload import to_f64
from tests import linear_norm
from tests.test_gpu_linear import CASES, inputs, on

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


@pytest.mark.parametrize("T,d,N,n,r", CASES + [
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
