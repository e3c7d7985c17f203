"""GPU tests of the training operators against their fp64 oracle, element by
element.

Tolerances.  u16 = 2^-8 is the rounding of a bf16 result (8-bit significand) and u32 = 2^-24 that
of an fp32 one.
 * Layer norm sums at most 16 + 28 * 8 terms in one chain, then a tree, in
   fp32: 512 u32 of the sum of magnitudes covers sums, statistics and the few
   operations behind them.
 * Logits: products of bf16 are exact in fp32; the tensor cores add with
   truncation, 16 products at a time, in runs of 1024: 64 additions, each off by at
   most 2^-23 of the magnitudes |x| |w| summed so far; the runs are added in fp32.
   So a logit is off by 2^-17 of |x| |w|.  A loss is a difference of two
   averages of logits, plus sums of exponentials with 2^-22 each.
 * Gradients: D is rounded to bf16 once (2^-8 of each entry), its logit error
   enters as a factor, and the sums of up to V (or T) terms are truncated as
   above: 2^-8 + 2^-12 of |D| |W| (or |D|^T |X|), then the bf16 rounding.
   Probabilities below fp32's normal range count as 0: 2^-126 per entry.
"""
import math

import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300.workload import to_f64
from oracle import train_ref

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def within(got, ref, bound):
    got = to_f64(got)
    assert got.shape == ref.shape
    off = np.abs(got - ref) - bound
    assert np.isfinite(got).all() and (off <= 0).all(), f"over the bound by {off.max()}, at {np.unravel_index(off.argmax(), off.shape)}"


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def same_bits(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b) if x is not None)


# ------------------------------------------------------------------ layer norm
def ln_inputs(rows, d, xt, wt, seed=0, shift=0.0):
    g = gen(seed)
    x = (torch.randn((rows, d), generator=g) * 2 + shift).to(xt)
    w, b = (1 + 0.3 * torch.randn(d, generator=g)).to(wt), (0.3 * torch.randn(d, generator=g)).to(wt)
    return x, w, b, torch.randn((rows, d), generator=g).to(xt)


def check_ln(train, x, w, b, dy, eps=1e-5):
    rows, d = x.shape
    X, Wt, B, DY = to_f64(x), to_f64(w), None if b is None else to_f64(b), to_f64(dy)
    y, mean, rstd = train.layer_norm_forward(x.to(DEV), w.to(DEV), None if b is None else b.to(DEV), eps)
    ry, rm, rr = train_ref.layer_norm(X, Wt, B, eps)
    e = 512 * U32
    amean = np.abs(X).mean(1)
    within(mean, rm, e * amean)
    # the mean's error shifts every element; relative to the spread it enters rstd squared
    dm = e * amean
    within(rstd, rr, rr * (e + (dm * rr) ** 2 + U32))
    n_off = (e * (np.abs(X - rm[:, None]) * rr[:, None]) + (dm * rr)[:, None] + 2 * U32 * np.abs(X) * rr[:, None])
    y_off = n_off * np.abs(Wt) + 4 * U32 * (np.abs(ry) + np.abs(0 if B is None else B))
    uy = U16 if x.dtype == torch.bfloat16 else U32
    within(y, ry, y_off + uy * (np.abs(ry) + y_off))

    saved = [mean, rstd]
    dx, dw, db = train.layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), *saved)
    sm, sr = to_f64(mean), to_f64(rstd)                                       # the backward's inputs
    rx, rw, rb = train_ref.layer_norm_backward(DY, X, Wt, sm, sr)
    n = np.abs(X - sm[:, None]) * sr[:, None]
    g = np.abs(DY * Wt)
    x_off = e * sr[:, None] * (g + g.mean(1, keepdims=True) + n * (g * n).mean(1, keepdims=True))
    within(dx, rx, x_off + uy * np.abs(rx))
    chain = (rows + 64) * U32                                                 # rows of one block, then 32 slices
    uw = U16 if w.dtype == torch.bfloat16 else U32
    w_off, b_off = (chain + 4 * U32) * (np.abs(DY) * n).sum(0), chain * np.abs(DY).sum(0)
    within(dw, rw, w_off + uw * np.abs(rw))
    within(db, rb, b_off + uw * np.abs(rb))
    again = train.layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), *saved)
    assert same_bits((dx, dw, db), again)
    assert same_bits((y, mean, rstd), train.layer_norm_forward(x.to(DEV), w.to(DEV), None if b is None else b.to(DEV), eps))


@pytest.mark.parametrize("xt,wt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 8), (3, 7), (2, 64), (5, 257), (33, 520), (1, 7168), (400, 1001),
                                    (1, 8192), (3, 8200), (2, 9001)])
def test_layer_norm(train, rows, d, xt, wt):
    check_ln(train, *ln_inputs(rows, d, xt, wt, seed=rows + d))


@pytest.mark.parametrize("rows,d,xt", [(1824, 256, torch.bfloat16), (1900, 1024, torch.float32),
                                       (1825, 2056, torch.bfloat16), (1830, 7168, torch.bfloat16),
                                       (930, 7168, torch.float32), (2001, 72, torch.bfloat16),
                                       (1999, 1001, torch.float32), (1830, 1003, torch.bfloat16),
                                       (1900, 2051, torch.float32), (2000, 4099, torch.bfloat16),
                                       (1850, 13, torch.bfloat16), (700, 8, torch.bfloat16), (513, 128, torch.float32),
                                       (3000, 200, torch.bfloat16), (10007, 64, torch.bfloat16)])
def test_layer_norm_many_rows(train, rows, d, xt):
    check_ln(train, *ln_inputs(rows, d, xt, torch.float32, seed=7))


# Rows whose shared memory comes to just 48 KB, of which the static part leaves a
# launch less without leave; the kernels of wider rows would ask for it first.
LN_48_KB = [(1830, 6144, torch.bfloat16), (9, 2048, torch.float32), (5, 2435, torch.bfloat16), (5, 2030, torch.float32)]


def ln_first_calls(queue):
    from mixture_experts_layer_19_gb300 import train
    failed = []
    for rows, d, xt in LN_48_KB:
        try:
            check_ln(train, *ln_inputs(rows, d, xt, torch.float32, seed=d))
        except Exception as e:
            failed.append(f"{rows} x {d} {xt}: {e}")
    queue.put(failed)


def test_layer_norm_near_48_kb_in_a_new_process():
    import torch.multiprocessing as mp
    ctx = mp.get_context("spawn")
    queue = ctx.Queue()
    child = ctx.Process(target=ln_first_calls, args=(queue,))
    child.start()
    try:
        assert queue.get(timeout=240) == []
    finally:
        child.join(60)
    assert child.exitcode == 0


def test_layer_norm_mean_far_from_zero_and_no_bias(train):
    """A difference of sums would lose the variance here: the mean is 300 spreads away."""
    x, w, _, dy = ln_inputs(40, 1024, torch.float32, torch.float32, seed=3, shift=600.0)
    check_ln(train, x, w, None, dy)
    x, w, _, dy = ln_inputs(1900, 1024, torch.float32, torch.float32, seed=4, shift=600.0)
    check_ln(train, x, w, None, dy)


def test_layer_norm_constant_rows(train):
    x = torch.full((3, 128), 2.5, dtype=torch.bfloat16, device=DEV)
    w, b = torch.ones(128, device=DEV), torch.full((128,), 0.25, device=DEV)
    y, mean, rstd = train.layer_norm_forward(x, w, b, 1e-5)
    assert torch.equal(mean, torch.full((3,), 2.5, device=DEV))
    assert (y == 0.25).all() and torch.allclose(rstd, torch.full((3,), 1e-5, device=DEV) ** -0.5)


@pytest.mark.parametrize("rows,d", [(7, 300), (2000, 512)])
def test_layer_norm_not_a_number_stays_in_its_row(train, rows, d):
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(rows, d, torch.bfloat16, torch.float32))
    good = train.layer_norm_forward(x, w, b)
    gdx, _, gdb = train.layer_norm_backward(dy, x, w, good[1], good[2])
    x2 = x.clone()
    x2[4, 3] = math.nan
    bad = train.layer_norm_forward(x2, w, b)
    dx, dw, db = train.layer_norm_backward(dy, x2, w, bad[1], bad[2])
    rest = torch.arange(rows, device=DEV) != 4
    assert same_bits([t[rest] for t in good], [t[rest] for t in bad]) and same_bits([gdx[rest], gdb], [dx[rest], db])
    assert bad[0][4].isnan().all() and dx[4].isnan().all() and dw.isnan().all()


def test_layer_norm_empty_leading_shape_and_skipped_outputs(train):
    w = torch.ones(16, device=DEV)
    y, mean, rstd = train.layer_norm_forward(torch.zeros((0, 16), dtype=torch.bfloat16, device=DEV), w)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = train.layer_norm_backward(y, y, w, mean, rstd)
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    x = torch.randn((2, 3, 16), device=DEV)
    y, mean, rstd = train.layer_norm_forward(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3)
    full = train.layer_norm_backward(x, x, w, mean, rstd)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        part = train.layer_norm_backward(x, x, w, mean, rstd, *need)
        for p, f, n in zip(part, full, need):
            assert (p is None) != n and (p is None or same_bits([p], [f]))


def test_layer_norm_autograd_matches_differences(train):
    """The gradient along a direction against differences of the kernel's own forward (fp32).  The
    forward's rounding, 512 u32 of the terms, is divided by 2h; the truncation is h^2 f''' / 6,
    taken from the same differences in 64 bits."""
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(6, 96, torch.float32, torch.float32, seed=5))
    x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    (train.layer_norm(x, w, b) * dy).sum().backward()
    h = 2.0 ** -6
    for leaf, pos in ((x, 0), (w, 1), (b, 2)):
        u = torch.sign(torch.randn(leaf.shape, generator=gen(9))).to(DEV)
        vals = [[t.detach() for t in (x, w, b)] for _ in range(2)]
        vals[0][pos], vals[1][pos] = leaf.detach() + h * u, leaf.detach() - h * u
        f = [(to_f64(train.layer_norm_forward(*v)[0]) * to_f64(dy)).sum() for v in vals]
        r = [(train_ref.layer_norm(*[to_f64(t) for t in v], 1e-5)[0] * to_f64(dy)).sum() for v in vals]
        slope = (to_f64(leaf.grad) * to_f64(u)).sum()
        ref = (f[0] - f[1]) / (2 * h)
        terms = (np.abs(to_f64(dy)) * (np.abs(to_f64(train.layer_norm_forward(x, w, b)[0])) + 1)).sum()
        rounding = 2 * 512 * U32 * terms / (2 * h)
        truncation = abs((r[0] - r[1]) / (2 * h) - slope)
        assert truncation < 0.05 * abs(slope) + 0.05 and abs(ref - slope) <= rounding + truncation


# ------------------------------------------------------------------ the loss head
def head_inputs(T, d, V, seed=0, scale=1.0):
    g = gen(seed)
    X = (torch.randn((T, d), generator=g) * scale).to(torch.bfloat16)
    W = (torch.randn((V, d), generator=g) / math.sqrt(d)).to(torch.bfloat16)
    return X, W, g


def labels_for(T, V, g, ignored=0.3, dtype=torch.int64):
    lab = torch.randint(0, V, (T,), generator=g)
    drop = torch.rand(T, generator=g) < ignored
    other = torch.tensor([-100, -1, V, 2 ** 31 - 1])[torch.randint(0, 4, (T,), generator=g)]
    return torch.where(drop, other, lab).to(dtype)


def check_head(train, X, W, dloss, targets, temp=1.0, labels=None, teacher=None, ids=None, piece=0):
    P, on, ent = targets
    Xd, Wd, g = X.to(DEV), W.to(DEV), dloss.to(DEV)
    if labels is not None:
        fwd = lambda: train.cross_entropy_forward(Xd, Wd, labels.to(DEV))                             # noqa: E731
        bwd = lambda lse, **k: train.cross_entropy_backward(g, Xd, Wd, labels.to(DEV), lse, **k)      # noqa: E731
    else:
        fwd = lambda: train.distill_forward(Xd, Wd, teacher.to(DEV), ids.to(DEV), temp)               # noqa: E731
        bwd = lambda lse, **k: train.distill_backward(g, Xd, Wd, teacher.to(DEV), ids.to(DEV), lse, temp, **k)  # noqa: E731
    loss, lse = fwd()
    X64, W64, G = to_f64(X), to_f64(W), to_f64(dloss)
    rl, rs = train_ref.head_loss(np.where(on[:, None], X64, 0), W64, P, on, ent, temp)
    # the largest |x| |w| of a row, in units of the loss
    dz = 2.0 ** -17 * (np.abs(np.where(on[:, None], X64, 0)) @ np.abs(W64).T).max(1) / temp + 2.0 ** -21
    within(lse, rs, on * (dz + 8 * U32 * np.abs(rs)))
    within(loss, rl, on * temp ** 2 * (2 * dz + 16 * U32 * (np.abs(rs) + np.abs(rl) + np.abs(ent))))
    dX, dW = bwd(lse, piece=piece)
    rX, rW, aX, aW = train_ref.head_gradients(G, np.where(on[:, None], X64, 0), W64, P, on, temp)
    c = U16 + 2.0 ** -12
    least = 2.0 ** -126 * (1 + temp * np.abs(G))
    within(dX, rX, c * aX + U16 * np.abs(rX) * (1 + c) + least[:, None] * np.abs(W64).sum(0))
    within(dW, rW, c * aW + U16 * np.abs(rW) * (1 + c) + (least[:, None] * np.abs(np.where(on[:, None], X64, 0))).sum(0))
    assert same_bits((loss, lse), fwd()) and same_bits((dX, dW), bwd(lse, piece=piece))
    only = bwd(lse, need_dW=False, piece=piece), bwd(lse, need_dX=False, piece=piece)
    assert only[0][1] is None and only[1][0] is None
    assert same_bits((dX, dW), (only[0][0], only[1][1]))
    return loss, lse, dX, dW


SIZES = [(1, 8, 1), (1, 64, 300), (5, 72, 257), (127, 64, 128), (128, 128, 256), (129, 136, 1000), (300, 520, 5003),
         (257, 1032, 777), (64, 2056, 300), (600, 256, 40), (1030, 64, 2500)]


@pytest.mark.parametrize("T,d,V", SIZES)
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_cross_entropy(train, T, d, V, dtype):
    X, W, g = head_inputs(T, d, V, seed=T + d + V)
    labels = labels_for(T, V, g, ignored=0.3 if dtype == torch.int64 else 0.0, dtype=dtype)
    P, on = train_ref.one_hot_targets(labels.numpy(), V)
    check_head(train, X, W, torch.full((T,), 1.0 / max(1, int(on.sum()))), (P, on, np.zeros(T)), labels=labels)


def test_cross_entropy_many_tokens(train):
    T, d, V = 40000, 64, 300
    X, W, g = head_inputs(T, d, V, seed=2)
    labels = labels_for(T, V, g, ignored=0.5)
    P, on = train_ref.one_hot_targets(labels.numpy(), V)
    check_head(train, X, W, torch.full((T,), 1.0 / int(on.sum())), (P, on, np.zeros(T)), labels=labels)


@pytest.mark.parametrize("piece", [256, 300, 512, 4096])
@pytest.mark.parametrize("T", [40, 300])
def test_cross_entropy_in_pieces_with_weights(train, T, piece):
    """Several pieces of the vocabulary, the last one short; every token has a weight of its own, some 0."""
    d, V = 264, 1100
    X, W, g = head_inputs(T, d, V, seed=piece)
    labels = labels_for(T, V, g)
    P, on = train_ref.one_hot_targets(labels.numpy(), V)
    weights = torch.randn(T, generator=g)
    weights[::7] = 0.0
    _, _, dX, _ = check_head(train, X, W, weights, (P, on, np.zeros(T)), labels=labels, piece=piece)
    assert (dX[::7] == 0).all()


def test_cross_entropy_large_logits(train):
    """Logits of several hundred: the softmax is one-hot for most rows."""
    X, W, g = head_inputs(50, 128, 900, seed=1, scale=100.0)
    labels = labels_for(50, 900, g)
    P, on = train_ref.one_hot_targets(labels.numpy(), 900)
    check_head(train, X, W, torch.ones(50), (P, on, np.zeros(50)), labels=labels)


def distill_targets(T, V, K, g, temp, dtype=torch.float32, messy=True):
    ids = torch.randint(0, V, (T, K), generator=g)                     # equal ids among them
    teacher = (3 * torch.randn((T, K), generator=g)).to(dtype)
    if messy:
        ids = torch.where(torch.rand((T, K), generator=g) < 0.2, torch.tensor([-1, V, -7])[ids % 3], ids)
        teacher = torch.where(torch.rand((T, K), generator=g) < 0.1, torch.tensor(-math.inf, dtype=dtype), teacher)
        ids[::5] = -1                                                  # rows without any entry
    return teacher, ids, train_ref.teacher_targets(to_f64(teacher), ids.numpy(), V, temp)


@pytest.mark.parametrize("T,d,V,K,temp", [(1, 8, 1, 1, 1.0), (3, 64, 40, 64, 2.0), (130, 72, 257, 5, 0.5),
                                          (300, 520, 5003, 20, 2.0), (64, 1032, 777, 33, 1.0), (9, 64, 3000, 1024, 4.0),
                                          (257, 128, 512, 2, 1.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distillation(train, T, d, V, K, temp, dtype):
    X, W, g = head_inputs(T, d, V, seed=T + K)
    teacher, ids, targets = distill_targets(T, V, K, g, temp, dtype, messy=T > 1)
    if dtype == torch.bfloat16:
        ids = ids.to(torch.int32)
    check_head(train, X, W, torch.full((T,), 1.0 / T), targets, temp, teacher=teacher, ids=ids)


def test_distillation_in_pieces(train):
    X, W, g = head_inputs(200, 136, 1500, seed=5)
    teacher, ids, targets = distill_targets(200, 1500, 12, g, 2.0)
    check_head(train, X, W, torch.randn(200, generator=g), targets, 2.0, teacher=teacher, ids=ids, piece=512)


def test_distillation_many_entries_in_one_tile(train):
    """All of a row's entries are neighbours in the vocabulary, in no order."""
    T, V, K = 140, 700, 100
    X, W, g = head_inputs(T, 64, V, seed=6)
    ids = torch.stack([250 + torch.randperm(K, generator=g) for _ in range(T)])
    teacher = torch.randn((T, K), generator=g)
    check_head(train, X, W, torch.ones(T), train_ref.teacher_targets(to_f64(teacher), ids.numpy(), V, 1.0),
               teacher=teacher, ids=ids)


def test_no_token_counts(train):
    X, W, _ = head_inputs(37, 64, 300)
    X[:] = math.nan
    lab = torch.full((37,), -100)
    Xd, Wd, g = X.to(DEV), W.to(DEV), torch.ones(37, device=DEV)
    loss, lse = train.cross_entropy_forward(Xd, Wd, lab.to(DEV))
    dX, dW = train.cross_entropy_backward(g, Xd, Wd, lab.to(DEV), lse)
    assert all((t == 0).all() for t in (loss, lse, dX, dW))
    u, ids = torch.full((37, 4), math.nan, device=DEV), torch.full((37, 4), -1, device=DEV)
    loss, lse = train.distill_forward(Xd, Wd, u, ids, 2.0)
    dX, dW = train.distill_backward(g, Xd, Wd, u, ids, lse, 2.0)
    assert all((t == 0).all() for t in (loss, lse, dX, dW))


def test_no_tokens(train):
    X, W = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV), torch.ones((300, 64), dtype=torch.bfloat16, device=DEV)
    lab, e = torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(0, device=DEV)
    loss, lse = train.cross_entropy_forward(X, W, lab)
    dX, dW = train.cross_entropy_backward(e, X, W, lab, lse)
    assert loss.shape == (0,) and dX.shape == (0, 64) and (dW == 0).all()


@pytest.mark.parametrize("T", [60, 300])
def test_masked_tokens_leave_no_trace(train, T):
    """What an ignored token's row, its upstream gradient and an unused entry hold changes no bit."""
    d, V, K = 128, 600, 6
    X, W, g = head_inputs(T, d, V, seed=8)
    labels = labels_for(T, V, g, ignored=0.4)
    off = (labels < 0) | (labels >= V)
    dl = torch.randn(T, generator=g)
    X2, dl2 = X.clone(), dl.clone()
    X2[off] = math.nan
    dl2[off] = math.inf
    Wd, lab = W.to(DEV), labels.to(DEV)
    a, b = train.cross_entropy_forward(X.to(DEV), Wd, lab), train.cross_entropy_forward(X2.to(DEV), Wd, lab)
    assert same_bits(a, b)
    ga = train.cross_entropy_backward(dl.to(DEV), X.to(DEV), Wd, lab, a[1])
    gb = train.cross_entropy_backward(dl2.to(DEV), X2.to(DEV), Wd, lab, a[1])
    assert same_bits(ga, gb)
    # a weight of 0 leaves a token out of the gradients too
    zero = dl.clone()
    zero[~off] *= (torch.arange(int((~off).sum())) % 2).float()
    X3 = X.clone()
    X3[zero == 0] = math.inf
    assert same_bits(train.cross_entropy_backward(zero.to(DEV), X.to(DEV), Wd, lab, a[1]),
                     train.cross_entropy_backward(zero.to(DEV), X3.to(DEV), Wd, lab, a[1]))
    teacher, ids, _ = distill_targets(T, V, K, g, 1.0)
    t2 = torch.where((ids < 0) | (ids >= V), torch.tensor(math.nan), teacher)
    a = train.distill_forward(X.to(DEV), Wd, teacher.to(DEV), ids.to(DEV))
    assert same_bits(a, train.distill_forward(X.to(DEV), Wd, t2.to(DEV), ids.to(DEV)))
    assert same_bits(train.distill_backward(dl.to(DEV), X.to(DEV), Wd, teacher.to(DEV), ids.to(DEV), a[1]),
                     train.distill_backward(dl.to(DEV), X.to(DEV), Wd, t2.to(DEV), ids.to(DEV), a[1]))


def test_not_a_number_in_a_token_that_counts_stays_in_its_row(train):
    T, d, V = 200, 64, 500
    X, W, g = head_inputs(T, d, V, seed=9)
    labels = torch.randint(0, V, (T,), generator=g)
    X2 = X.clone()
    X2[77, 5] = math.nan
    X2[78, 5] = math.inf
    rest = torch.ones(T, dtype=torch.bool)
    rest[77:79] = False
    a, b = (train.cross_entropy_forward(x.to(DEV), W.to(DEV), labels.to(DEV)) for x in (X, X2))
    assert same_bits([t[rest.to(DEV)] for t in a], [t[rest.to(DEV)] for t in b]) and b[0][77:79].isnan().all()
    dl = torch.ones(T, device=DEV)
    ga, gb = (train.cross_entropy_backward(dl, x.to(DEV), W.to(DEV), labels.to(DEV), f[1]) for x, f in ((X, a), (X2, b)))
    assert same_bits([ga[0][rest.to(DEV)]], [gb[0][rest.to(DEV)]]) and gb[0][77].isnan().all()
    dl[3] = math.nan                                                    # an upstream gradient
    gc = train.cross_entropy_backward(dl, X.to(DEV), W.to(DEV), labels.to(DEV), a[1])
    assert gc[0][3].isnan().all() and not gc[0][4:].isnan().any() and gc[1].isnan().all()


def test_one_entry_with_probability_one_is_cross_entropy(train):
    T, d, V = 150, 128, 900
    X, W, g = head_inputs(T, d, V, seed=10)
    labels = labels_for(T, V, g).clamp(max=V)
    Xd, Wd, lab = X.to(DEV), W.to(DEV), labels.to(DEV)
    dl = torch.randn(T, generator=g).to(DEV)
    a = train.cross_entropy_forward(Xd, Wd, lab)
    b = train.distill_forward(Xd, Wd, torch.zeros((T, 1), device=DEV), lab[:, None].contiguous())
    assert same_bits(a, b)
    assert same_bits(train.cross_entropy_backward(dl, Xd, Wd, lab, a[1]),
                     train.distill_backward(dl, Xd, Wd, torch.zeros((T, 1), device=DEV), lab[:, None].contiguous(), a[1]))


@pytest.mark.parametrize("kind", ["labels", "teacher"])
def test_head_autograd_matches_differences(train, kind):
    """Along a direction, against differences of the kernel's own loss.  X and W lie on a grid on
    which a step of 1/64 is exact in bf16.  The forward's error (2^-17 of |x| |w| per logit, twice per
    loss) is divided by 2h; the truncation is taken from the same differences in 64 bits; the gradient's
    own rounding is that of its elements."""
    T, d, V, K, temp, h = 20, 32, 150, 4, 2.0, 1.0 / 64
    g = gen(11)
    X = (torch.randint(-30, 31, (T, d), generator=g) / 64).to(torch.bfloat16).to(DEV).requires_grad_()
    W = (torch.randint(-30, 31, (V, d), generator=g) / 64).to(torch.bfloat16).to(DEV).requires_grad_()
    weights = torch.randn(T, generator=g).to(DEV)
    if kind == "labels":
        temp, labels = 1.0, labels_for(T, V, g)
        loss = lambda x, w: train.linear_cross_entropy(x, w, labels.to(DEV))                                # noqa: E731
        P, on = train_ref.one_hot_targets(labels.numpy(), V)
        ent = np.zeros(T)
    else:
        teacher, ids, (P, on, ent) = distill_targets(T, V, K, g, temp)
        loss = lambda x, w: train.linear_distillation(x, w, teacher.to(DEV), ids.to(DEV), temp)            # noqa: E731
    (loss(X, W) * weights).sum().backward()
    G = to_f64(weights)
    for leaf in (X, W):
        u = torch.sign(torch.randn(leaf.shape, generator=gen(12))).to(DEV).to(torch.bfloat16)
        pts = []
        for sgn in (1, -1):
            v = (leaf.detach() + sgn * h * u)
            pts.append((v, W.detach()) if leaf is X else (X.detach(), v))
        f = [(to_f64(loss(*p)) * G).sum() for p in pts]
        r = [(train_ref.head_loss(*[to_f64(t) for t in p], P, on, ent, temp)[0] * G).sum() for p in pts]
        rX, rW, aX, aW = train_ref.head_gradients(G, to_f64(X), to_f64(W), P, on, temp)
        want = (rX if leaf is X else rW)
        mag = (aX if leaf is X else aW)
        slope = (to_f64(leaf.grad) * to_f64(u)).sum()
        truncation = abs((r[0] - r[1]) / (2 * h) - (want * to_f64(u)).sum())
        dz = 2.0 ** -17 * (np.abs(to_f64(X)) @ np.abs(to_f64(W)).T).max() + 2.0 ** -18
        rounding = 2 * temp ** 2 * 2 * dz * np.abs(G).sum() / (2 * h) + (2 * U16 * (mag + np.abs(want))).sum()
        assert abs((f[0] - f[1]) / (2 * h) - slope) <= rounding + truncation
        assert abs(truncation) < 0.1 * abs((want * to_f64(u)).sum()) + 0.1


def test_head_refuses_on_the_gpu(train):
    from mixture_experts_layer_19_gb300 import moe
    X, W = torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV), torch.zeros((10, 16), dtype=torch.bfloat16, device=DEV)
    lab, st = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    buf = torch.zeros(4 * 16 + 1, dtype=torch.bfloat16, device=DEV)
    u, ids = torch.zeros((4, 2), device=DEV), torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    for call in (lambda: train.cross_entropy_forward(buf[1:].view(4, 16), W, lab),              # 2-byte aligned
                 lambda: train.cross_entropy_forward(X.t().contiguous().t(), W, lab),           # strides
                 lambda: train.cross_entropy_forward(X, W.cpu(), lab),
                 lambda: train.cross_entropy_forward(X, W, lab.cpu()),
                 lambda: train.layer_norm_forward(buf[1:].view(4, 16), torch.ones(16, device=DEV)),
                 lambda: train.layer_norm_forward(X[:, ::2], torch.ones(8, device=DEV)),
                 lambda: train.distill_forward(X, W, u.t().contiguous().t(), ids)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: train.cross_entropy_forward(X[:, :12].contiguous(), W[:, :12].contiguous(), lab),   # d = 12
                 lambda: train.cross_entropy_forward(X, W[:0], lab),
                 lambda: train.distill_forward(X, W, u, ids, temperature=0.0),
                 lambda: train.distill_forward(X, W, u[:, :0].contiguous(), ids[:, :0].contiguous()),
                 lambda: train.distill_forward(X, W, torch.zeros((4, 1025), device=DEV),
                                               torch.zeros((4, 1025), dtype=torch.int64, device=DEV)),
                 lambda: train.cross_entropy_backward(st, X, W, lab, st, piece=-1)):
        with pytest.raises(moe.MoEError):
            call()
    # a workspace that is too small is refused by the C entry point
    import ctypes
    cfg = moe.moe_head_config_t(4, 10, 16, 0, 1.0, 1, 0, 0, 0, 0)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    st4 = moe.lib().moe_cross_entropy_forward(ctypes.byref(cfg), X.data_ptr(), W.data_ptr(), lab.data_ptr(),
                                              st.data_ptr(), st.data_ptr(), ws.data_ptr(), 64, None, None)
    assert st4 == moe.MOE_ERR_INVALID_ARG and b"workspace" in moe.lib().moe_last_error()


def test_another_stream_and_graph_replay(train):
    T, d, V = 200, 256, 1000
    X, W, g = head_inputs(T, d, V, seed=13)
    labels = labels_for(T, V, g)
    Xd, Wd, lab, dl = X.to(DEV), W.to(DEV), labels.to(DEV), torch.randn(T, generator=g).to(DEV)
    w = torch.ones(d, device=DEV)

    def step():
        y, mean, rstd = train.layer_norm_forward(Xd, w)
        loss, lse = train.cross_entropy_forward(y, Wd, lab)
        dX, dW = train.cross_entropy_backward(dl, y, Wd, lab, lse)
        return (loss, dX, dW, *train.layer_norm_backward(dX, Xd, w, mean, rstd))

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, mean, rstd = train.layer_norm_forward(Xd, w, stream=side)
    loss, lse = train.cross_entropy_forward(y, Wd, lab, stream=side)
    dX, dW = train.cross_entropy_backward(dl, y, Wd, lab, lse, stream=side)
    side.synchronize()
    assert same_bits((loss, dX, dW), ref[:3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(ref, out)


def test_offsets_past_32_bits(train):
    """W has 2.5e9 elements: the last vocabulary entries lie past 2^31 elements and 2^32 bytes."""
    T, d, V = 3, 8192, 300000
    W = torch.zeros((V, d), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    W[-1000:] = torch.randn((1000, d), generator=g, device=DEV).to(torch.bfloat16) / 64
    X = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    lab = torch.tensor([V - 1, 5, V - 700], device=DEV)
    loss, lse = train.cross_entropy_forward(X, W, lab)
    z = X.double() @ W[-1000:].double().T                                  # the other logits are 0
    ref = torch.logsumexp(torch.cat([z, torch.full((T, 1), math.log(V - 1000.0), device=DEV).double()], 1), 1)
    zl = torch.stack([z[0, -1], z.new_zeros(()), z[2, -700]])
    dz = 2.0 ** -17 * float((X.double().abs() @ W[-1000:].double().abs().T).max()) + 2.0 ** -18
    assert (lse.double() - ref).abs().max() <= dz and (loss.double() - (ref - zl)).abs().max() <= 2 * dz
    dX, dW = train.cross_entropy_backward(torch.ones(T, device=DEV), X, W, lab, lse)
    D = torch.exp(z - ref[:, None])
    D[0, -1] -= 1
    D[2, -700] -= 1
    c = U16 + 2.0 ** -12
    want, mag = D.T @ X.double(), D.abs().T @ X.double().abs()
    assert ((dW[-1000:].double() - want).abs() <= c * mag + U16 * want.abs() * (1 + c)).all()
    want, mag = D @ W[-1000:].double(), D.abs() @ W[-1000:].double().abs()
    assert ((dX.double() - want).abs() <= c * mag + U16 * want.abs() * (1 + c)).all()
    del W, dW
    rows = 270000
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn((2, d), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.ones(d, device=DEV)
    y, mean, rstd = train.layer_norm_forward(x, w)
    few = train.layer_norm_forward(x[-2:].clone(), w)
    assert (y[:-2] == 0).all() and ((y[-2:] - few[0]).abs() <= 2 * U16 * few[0].abs() + 1e-6).all()
    assert ((mean[-2:] - few[1]).abs() <= 1e-6).all()


def test_device_wait_expires_cleanly(train):
    """The producers issue nothing, so the waits run out: the status says so and the context stays usable."""
    from mixture_experts_layer_19_gb300 import moe
    for T in (40, 300):                                                    # single CTAs and CTA pairs
        X, W, g = head_inputs(T, 128, 600, seed=14)
        Xd, Wd, lab = X.to(DEV), W.to(DEV), torch.randint(0, 600, (T,), generator=g).to(DEV)
        ref = train.cross_entropy_forward(Xd, Wd, lab)
        train.cross_entropy_forward(Xd, Wd, lab, wait_timeout_ns=20_000_000, debug_flags=train.MOE_DEBUG_STALL_TEST)
        assert train.device_status(0) == moe.MOE_ERR_TIMEOUT
        assert train.device_status(0) == 0
        assert same_bits(ref, train.cross_entropy_forward(Xd, Wd, lab))


def test_modules_train(train):
    """LayerNorm -> LMHead under an optimiser: the loss falls, for labels and for a teacher."""
    torch.manual_seed(0)
    T, d, V = 256, 128, 500
    x = torch.randn((T, d), device=DEV).to(torch.bfloat16)
    lab = torch.randint(0, V, (T,), device=DEV)
    norm, head = train.LayerNorm(d), train.LMHead(d, V)
    opt = torch.optim.SGD([*norm.parameters(), *head.parameters()], lr=2.0)
    losses = []
    for i in range(30):
        f = norm(x)
        loss = head(f, lab).mean()
        if i >= 15:
            loss = head.distill(f, torch.zeros((T, 2), device=DEV), torch.stack([lab, lab], 1), 2.0).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    assert losses[14] < 0.7 * losses[0] and losses[29] < losses[15]


def test_example_step_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(["--tokens", "256", "--width", "256", "--ffn", "256", "--experts", "8", "--vocab", "1000",
                       "--steps", "12"])
    assert losses["cross entropy"][-1] < losses["cross entropy"][0]
    assert losses["distillation"][-1] < losses["distillation"][0]
