"""GPU tests of the loss head where its gradient is a small difference: tokens
that the model already predicts well, at a width where the tensor cores'
truncation shows.

Tolerances.  Both directions add a logit's products in the same runs of at most 1024, 16 products at
a time: each of the 64 additions is off by at most 2^-23 of what the run has summed so far, on average
half of the run's |x| |w|, so a logit is off by delta = 2^-18 of |x| |w| (runs are added in fp32: 8 u32).
 * The softmax is taken over the same logits: q_v = exp(z_v) / sum exp(z_u) moves by at most
   q_v sum_u q_u |delta_v - delta_u| <= 2 delta q_v (1 - q_v), and the loss of a label by 2 delta (1 - q).
 * What is not shared is rounding around the log-sum-exp, which is kept in fp32: eps = 4 u32 |lse|, plus
   2^-20 for the exponentials and sums.  It moves every q_v by q_v eps, and the loss by eps.
 * D = q - p is rounded to bf16 (2^-8 of |D|, p itself to 2^-20), and the sums dX = D W and dW = D^T X
   are truncated (63 additions of 2^-23, 2^-17 of |D| |W|) and rounded to bf16.
"""
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


def over(got, ref, bound):
    """By how many times the bound `got` is off at most."""
    got = to_f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    return float((np.abs(got - ref) / bound).max())


def confident_inputs(T, d, V, seed, margins, sharp=None):
    """Logits of 20 to 50 times `scale`; each token's label leads the others by one of `margins`."""
    g = gen(seed)
    u = torch.sign(torch.randn(d, generator=g))
    W = ((0.7 * torch.randn((V, d), generator=g) + 0.35 * u) / d ** 0.5).to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), generator=g)
    lead = torch.linspace(*margins, T)[:, None] / 0.49
    X = 0.8 * u + lead * W[labels].float()
    if sharp is not None:                                  # a second entry beside the label, half as far ahead
        X = X + sharp * lead * W[(labels + 1) % V].float()
    return X.to(torch.bfloat16), W, labels, g


def check(train, X, W, P, on, ent, temp, fwd, bwd, G):
    T = X.shape[0]
    X64, W64 = to_f64(X), to_f64(W)
    rl, rs = train_ref.head_loss(X64, W64, P, on, ent, temp)
    z = X64 @ W64.T / temp
    q = np.exp(z - rs[:, None])
    delta = ((2.0 ** -18 + 8 * U32) * (np.abs(X64) @ np.abs(W64).T).max(1) / temp)[:, None]
    eps = (4 * U32 * np.abs(rs) + 2.0 ** -20)[:, None]
    loss, lse = fwd()
    rest = (P * (1 - q)).sum(1)
    worst = {"lse": over(lse, rs, (delta + eps)[:, 0]),
             "loss": over(loss, rl, temp ** 2 * (2 * delta[:, 0] * rest + eps[:, 0] * (1 + np.abs(ent))))}
    dX, dW = bwd(lse)
    g = temp * to_f64(G)[:, None]
    D = g * (q - P)
    dD = np.abs(g) * ((U16 + 2.0 ** -17) * np.abs(q - P) + 2 * delta * q * (1 - q) + q * eps + 2.0 ** -20 * P)
    for name, got, ref, off in (("dX", dX, D @ W64, dD @ np.abs(W64)), ("dW", dW, D.T @ X64, dD.T @ np.abs(X64))):
        worst[name] = over(got, ref, off + U16 * (np.abs(ref) + off))
    assert all(v <= 1 for v in worst.values()), worst


@pytest.mark.parametrize("T", [7, 40, 100, 300])
@pytest.mark.parametrize("d", [2056, 7168])
def test_cross_entropy_of_well_predicted_tokens(train, T, d):
    V = 1000
    X, W, labels, g = confident_inputs(T, d, V, T, (9.0, 18.0))
    P, on = train_ref.one_hot_targets(labels.numpy(), V)
    G = torch.rand(T, generator=g) + 0.5
    Xd, Wd, lab, Gd = X.to(DEV), W.to(DEV), labels.to(DEV), G.to(DEV)
    check(train, X, W, P, on, np.zeros(T), 1.0, lambda: train.cross_entropy_forward(Xd, Wd, lab),
          lambda lse: train.cross_entropy_backward(Gd, Xd, Wd, lab, lse), G)


@pytest.mark.parametrize("T", [7, 40, 100, 300])
@pytest.mark.parametrize("temp", [1.0, 2.0])
def test_distillation_of_a_student_that_agrees(train, T, temp):
    """The teacher's entries are the student's own largest logits, slightly off."""
    V, d, K = 1000, 7168, 6
    X, W, _, g = confident_inputs(T, d, V, T + 1, (12.0, 20.0), sharp=0.9)
    top = torch.topk(X.double() @ W.double().T, K, dim=1)
    teacher = (top.values + 0.01 * torch.randn((T, K), generator=g)).float()
    ids = top.indices
    P, on, ent = train_ref.teacher_targets(to_f64(teacher), ids.numpy(), V, temp)
    G = torch.rand(T, generator=g) + 0.5
    Xd, Wd, td, idd, Gd = X.to(DEV), W.to(DEV), teacher.to(DEV), ids.to(DEV), G.to(DEV)
    check(train, X, W, P, on, ent, temp, lambda: train.distill_forward(Xd, Wd, td, idd, temp),
          lambda lse: train.distill_backward(Gd, Xd, Wd, td, idd, lse, temp), G)


@pytest.mark.parametrize("T", [1, 16, 40, 100, 300])
@pytest.mark.parametrize("d", [520, 1032, 7168])
def test_vocabulary_of_one_has_no_gradient(train, T, d):
    """D = exp(z - lse) - 1 with lse = z + log s, where s is 1 to within 2^-21: for z past 16 that is less than
    half a unit of its last place, so lse is z, if the two directions' logits agree to the bit, and D is 0."""
    g = gen(T + d)
    X = (torch.rand((T, d), generator=g) + 0.1).to(torch.bfloat16).to(DEV)
    W = ((torch.rand((1, d), generator=g) + 0.1) * (64 / d)).to(torch.bfloat16).to(DEV)
    labels = torch.zeros(T, dtype=torch.int64, device=DEV)
    loss, lse = train.cross_entropy_forward(X, W, labels)
    dX, dW = train.cross_entropy_backward(torch.ones(T, device=DEV), X, W, labels, lse)
    assert (lse > 16).all() and all((t == 0).all() for t in (loss, dX, dW))


@pytest.mark.parametrize("T,d,V,piece", [(300, 7168, 20000, 1024), (300, 1032, 4000, 256), (40, 2056, 5000, 512)])
def test_logits_do_not_depend_on_the_tiles(train, T, d, V, piece):
    """dW of a piece is D^T X of its own columns: pieces, and with them CTA pairs and tile widths, change no bit."""
    X, W, labels, g = confident_inputs(T, d, V, T, (0.0, 12.0))
    Xd, Wd, lab, G = X.to(DEV), W.to(DEV), labels.to(DEV), torch.rand(T, generator=g).to(DEV)
    _, lse = train.cross_entropy_forward(Xd, Wd, lab)
    whole = train.cross_entropy_backward(G, Xd, Wd, lab, lse)
    cut = train.cross_entropy_backward(G, Xd, Wd, lab, lse, piece=piece)
    assert torch.equal(whole[1], cut[1])
