"""Host-side refusals of the differentiable training operators (no GPU): ValueError before any library call."""
import pytest
import torch


@pytest.fixture
def train(monkeypatch):
    from mixture_experts_layer_19_gb300 import moe, train

    class NoCalls:
        def __getattr__(self, name):
            raise AssertionError(f"library called: {name}")

    monkeypatch.setattr(moe, "lib", lambda: NoCalls())
    return train


def test_differentiable_operators_refuse(train):
    T, d, V, K = 4, 16, 10, 3
    X, W = torch.zeros((T, d), dtype=torch.bfloat16), torch.zeros((V, d), dtype=torch.bfloat16)
    X3, lab = X.view(2, 2, d), torch.zeros(T, dtype=torch.int64)
    u, ids = torch.zeros((T, K)), torch.zeros((T, K), dtype=torch.int64)
    calls = [
        lambda: train.layer_norm(None, torch.ones(d)),
        lambda: train.layer_norm(X, None),
        lambda: train.layer_norm(X, torch.ones(d)),                                # not on a GPU
        lambda: train.linear_cross_entropy(None, W, lab),
        lambda: train.linear_cross_entropy(X, W, None),
        lambda: train.linear_cross_entropy(X, None, lab),
        lambda: train.linear_cross_entropy(X, W, lab[:3]),
        lambda: train.linear_cross_entropy(X, W, lab),                             # not on a GPU
        lambda: train.linear_cross_entropy(X3, W, None),
        lambda: train.linear_cross_entropy(X3, W, lab),                            # [4] for [2, 2]
        lambda: train.linear_cross_entropy(X3, W, lab.view(2, 2, 1)),
        lambda: train.linear_distillation(None, W, u, ids),
        lambda: train.linear_distillation(X, W, None, ids),
        lambda: train.linear_distillation(X, W, u, None),
        lambda: train.linear_distillation(X, W, u, ids[:, :2]),
        lambda: train.linear_distillation(X3, W, u, ids),
        lambda: train.linear_distillation(X3, W, u.view(2, 2, K), None),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
