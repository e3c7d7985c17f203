"""CPU tests of the training operators' fp64 oracle: gradients against
central differences, brute force on tiny shapes, and the masked cases."""
import numpy as np
import pytest

from oracle import train_ref


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        dn = f()
        x[i] = keep
        g[i] = (up - dn) / (2 * h)
    return g


# central differences at h = 1e-6 in fp64: truncation h^2 f''' / 6 and cancellation
# 1e-16 |f| / h, both below 1e-8 for these sizes
TOL = 1e-7


def test_layer_norm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    x, w, b, dy = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=7), rng.normal(size=(3, 7))

    def f():
        return (train_ref.layer_norm(x, w, b, 1e-5)[0] * dy).sum()

    _, mean, rstd = train_ref.layer_norm(x, w, b, 1e-5)
    dx, dw, db = train_ref.layer_norm_backward(dy, x, w, mean, rstd)
    for got, arr in ((dx, x), (dw, w), (db, b)):
        assert np.abs(got - _differences(f, arr)).max() < TOL


def test_layer_norm_statistics():
    x = np.random.default_rng(1).normal(size=(4, 50)) * 3 + 2
    y, mean, rstd = train_ref.layer_norm(x, np.ones(50), None, 0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-12) and np.allclose(y.var(-1), 1)
    assert np.allclose(mean, x.mean(-1)) and np.allclose(rstd, 1 / x.std(-1))


@pytest.mark.parametrize("kind", ["labels", "teacher"])
def test_head_gradients_match_differences(kind):
    rng = np.random.default_rng(2)
    T, d, V, K, temp = 4, 5, 9, 3, 2.0
    X, W, g = rng.normal(size=(T, d)), rng.normal(size=(V, d)), rng.normal(size=T)
    if kind == "labels":
        temp = 1.0
        P, on = train_ref.one_hot_targets(np.array([3, -100, 8, 0]), V)
        ent = np.zeros(T)
    else:
        ids = np.array([[1, 4, 7], [0, 0, 5], [-1, 9, -1], [8, -1, 2]])      # equal ids, none in use, one unused
        P, on, ent = train_ref.teacher_targets(rng.normal(size=(T, K)), ids, V, temp)
        assert list(on) == [True, True, False, True]

    def f():
        return (train_ref.head_loss(X, W, P, on, ent, temp)[0] * g).sum()

    dX, dW, _, _ = train_ref.head_gradients(g, X, W, P, on, temp)
    assert np.abs(dX - _differences(f, X)).max() < TOL * 10
    assert np.abs(dW - _differences(f, W)).max() < TOL * 10


def test_head_loss_by_brute_force():
    X, W = np.array([[1.0, 2.0]]), np.array([[0.5, 0.0], [0.0, 1.0], [-1.0, 0.5]])
    z = [0.5, 2.0, 0.0]
    P, on = train_ref.one_hot_targets(np.array([1]), 3)
    loss, lse = train_ref.head_loss(X, W, P, on, np.zeros(1))
    total = sum(np.exp(v) for v in z)
    assert np.isclose(lse[0], np.log(total)) and np.isclose(loss[0], -np.log(np.exp(2.0) / total))
    # a teacher that agrees with the student over the whole vocabulary costs nothing
    P, on, ent = train_ref.teacher_targets(np.array([z]), np.array([[0, 1, 2]]), 3, 2.0)
    loss, _ = train_ref.head_loss(X, W, P, on, ent, 2.0)
    assert abs(loss[0]) < 1e-12


def test_tokens_without_a_loss_take_part_in_nothing():
    rng = np.random.default_rng(3)
    X, W = rng.normal(size=(3, 4)), rng.normal(size=(6, 4))
    X[1] = np.nan
    P, on = train_ref.one_hot_targets(np.array([2, 6, 5]), 6)                # 6 is outside the vocabulary
    loss, lse = train_ref.head_loss(X, W, P, on, np.zeros(3))
    dX, dW, _, _ = train_ref.head_gradients(np.ones(3), X, W, P, on)
    assert loss[1] == 0 and lse[1] == 0 and (dX[1] == 0).all()
    assert np.isfinite(loss).all() and np.isfinite(dW).all()
