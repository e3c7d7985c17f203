"""Host-side checks of the training operators (no GPU): argument refusals come
as ValueError before any library call, and the C entry points refuse bad
sizes and pointers synchronously."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_19_gb300 import build as b
    b.build()
    from mixture_experts_layer_19_gb300 import moe
    return moe.load_library()


@pytest.fixture
def train(monkeypatch):
    from mixture_experts_layer_19_gb300 import moe, train

    class NoCalls:
        def __getattr__(self, name):
            raise AssertionError(f"library called: {name}")

    monkeypatch.setattr(moe, "lib", lambda: NoCalls())
    return train


bf = torch.bfloat16


def test_layer_norm_refusals(train):
    x, w = torch.zeros((3, 16), dtype=bf), torch.ones(16)
    st = torch.zeros(3)
    calls = [
        lambda: train.layer_norm_forward(None, w),
        lambda: train.layer_norm_forward(x, None),
        lambda: train.layer_norm_forward(x.half(), w),
        lambda: train.layer_norm_forward(x, w.double()),
        lambda: train.layer_norm_forward(x, w[:8]),
        lambda: train.layer_norm_forward(x[:, :0], w[:0]),
        lambda: train.layer_norm_forward(torch.zeros((), dtype=bf), w),
        lambda: train.layer_norm_forward(x, w, torch.zeros(16, dtype=bf)),       # bias of another type
        lambda: train.layer_norm_forward(x, w),                                   # not on a GPU
        lambda: train.layer_norm_backward(x.float(), x, w, st, st),
        lambda: train.layer_norm_backward(x[:2], x, w, st, st),
        lambda: train.layer_norm_backward(x, x, w, st.to(bf), st),
        lambda: train.layer_norm_backward(x, x, w, st, st[:2]),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_head_refusals(train):
    T, d, V, K = 4, 16, 10, 3
    X, W = torch.zeros((T, d), dtype=bf), torch.zeros((V, d), dtype=bf)
    lab, g = torch.zeros(T, dtype=torch.int64), torch.zeros(T)
    u, ids = torch.zeros((T, K)), torch.zeros((T, K), dtype=torch.int32)
    calls = [
        lambda: train.cross_entropy_forward(X.float(), W, lab),
        lambda: train.cross_entropy_forward(X, W.float(), lab),
        lambda: train.cross_entropy_forward(X[0], W, lab),
        lambda: train.cross_entropy_forward(X, W[:, :8], lab),
        lambda: train.cross_entropy_forward(X, W, lab[:3]),
        lambda: train.cross_entropy_forward(X, W, lab.float()),
        lambda: train.cross_entropy_forward(X, W, None),
        lambda: train.cross_entropy_forward(X, W, lab),                           # not on a GPU
        lambda: train.cross_entropy_backward(g.double(), X, W, lab, g),
        lambda: train.cross_entropy_backward(g, X, W, lab, g[:2]),
        lambda: train.distill_forward(X, W, u.double(), ids),
        lambda: train.distill_forward(X, W, u[:3], ids[:3]),
        lambda: train.distill_forward(X, W, u, ids[:, :2]),
        lambda: train.distill_forward(X, W, u, ids.float()),
        lambda: train.distill_backward(g, X, W, u, ids, None),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_c_entry_points_refuse_bad_sizes(lib):
    from mixture_experts_layer_19_gb300.moe import moe_head_config_t
    n = ctypes.c_size_t()
    good = dict(T=4, V=10, d=16, K=3, temperature=1.0, ids_int64=1, teacher_bf16=0, piece=0, wait_timeout_ns=0,
                debug_flags=0)
    bad = [dict(T=-1), dict(T=(1 << 20) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(d=0), dict(d=12),
           dict(d=(1 << 16) + 8), dict(K=0), dict(K=1025), dict(temperature=0.0), dict(temperature=float("inf")),
           dict(temperature=float("nan")), dict(piece=-1), dict(wait_timeout_ns=-1)]
    for change in bad:
        kw = {**good, **change}
        cfg = moe_head_config_t(*[kw[f[0]] for f in moe_head_config_t._fields_])
        st = lib.moe_head_workspace_bytes(ctypes.byref(cfg), 1, 1, ctypes.byref(n))
        assert st in (1, 2), (change, st)
        assert lib.moe_last_error()
        assert lib.moe_distill_forward(ctypes.byref(cfg), *[None] * 7, 0, None, None) in (1, 2), change
    assert lib.moe_head_workspace_bytes(None, 0, 0, ctypes.byref(n)) == 1
    cfg = moe_head_config_t(*[good[f[0]] for f in moe_head_config_t._fields_])
    assert lib.moe_head_workspace_bytes(ctypes.byref(cfg), 0, 0, None) == 1
    # null and misaligned pointers are argument errors before anything touches a GPU
    assert lib.moe_cross_entropy_forward(ctypes.byref(cfg), *[None] * 6, 0, None, None) == 1
    assert lib.moe_cross_entropy_forward(ctypes.byref(cfg), 8, 16, 16, 16, 16, 256, 1 << 20, None, None) == 1
    cfg.T = 0
    assert lib.moe_cross_entropy_forward(ctypes.byref(cfg), *[None] * 6, 0, None, None) == 0


def test_layer_norm_c_entry_points_refuse_bad_sizes(lib):
    fwd = lib.moe_layer_norm_forward
    assert fwd(None, None, None, -1, 8, 0, 0, 1e-5, None, None, None, None) == 1
    assert fwd(None, None, None, 4, 0, 0, 0, 1e-5, None, None, None, None) == 1
    assert fwd(None, None, None, 4, (1 << 20) + 1, 0, 0, 1e-5, None, None, None, None) == 1
    assert fwd(16, 16, None, 4, 8, 0, 0, -1.0, 16, 16, 16, None) == 1
    assert fwd(16, 16, None, 4, 8, 0, 0, float("nan"), 16, 16, 16, None) == 1
    assert fwd(None, 16, None, 4, 8, 0, 0, 1e-5, 16, 16, 16, None) == 1
    assert fwd(18, 16, None, 4, 8, 0, 0, 1e-5, 16, 16, 16, None) == 1
    assert fwd(None, None, None, 0, 8, 0, 0, 1e-5, None, None, None, None) == 0
    bwd = lib.moe_layer_norm_backward
    assert bwd(16, 16, 16, 16, 16, 4, 8, 0, 0, 16, 16, 16, None, 0, None) == 1      # workspace missing
    assert bwd(16, 16, 16, None, 16, 4, 8, 0, 0, 16, None, None, None, 0, None) == 1
    assert lib.moe_layer_norm_workspace_bytes(4, 8, None) == 1
