"""The bound in norm that fp32 results of a projection are held to on the GPU tells them from results without what makes
them exact: sums that end every 512 products, and the third part of u.  The mistakes are planted in the restatement."""
import numpy as np
import pytest

from tests import linear_norm as ln


def exact(X, W, A, B):
    X, W, A, B = (t.astype(np.float64) for t in (X, W, A, B))
    return X @ W.T + X @ A.T @ B.T


def inputs(T, d, N, r, w=1.0):
    g = np.random.default_rng(d + r)
    f = lambda *s, by=1.0: ln.bf16((by * g.standard_normal(s)).astype(np.float32))                   # noqa: E731
    return f(T, d), f(N, d, by=w / d ** 0.5), f(r, d, by=d ** -0.5), f(N, r)


@pytest.mark.parametrize("d", [4096, 8192])
def test_sums_without_an_end_show(d):
    s = inputs(8, d, 200, 16)
    ref = exact(*s)
    assert ln.off(ln.linear(*s), ref) < ln.tolerance(16) < ln.off(ln.linear(*s, every=1 << 20), ref)


@pytest.mark.parametrize("d,r", [(512, 16), (2048, 64)])
def test_a_missing_third_part_shows(d, r):
    s = inputs(16, d, 200, r, w=2.0 ** -12)
    ref = exact(*s)
    three, two = (ln.off(ln.linear(*s, parts=p), ref) for p in (3, 2))
    assert three < ln.tolerance(r) < two
