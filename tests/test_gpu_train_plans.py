"""GPU tests of the loss head's tile plans: CTA pairs with several tiles each, for labels and for teachers;
tiles of 128 and 192 columns; the default cut of the vocabulary into pieces; the expired wait of a pair.  Each
asserts the plan it is about.

The reference is the fp64 statement of oracle/train_ref.py, written in torch to run on the GPU; the bounds
are those of tests/test_gpu_train.py."""
import pytest
import torch

from tests.test_gpu_train import distill_targets, head_inputs, labels_for, same_bits

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


def bounded(got, ref, bound, what):
    off = (got.double() - ref).abs() - bound
    assert torch.isfinite(got).all() and (off <= 0).all(), f"{what}: over the bound by {float(off.max())}"


def check(fwd, bwd, X, W, P, on, ent, temp, G):
    """P [T, V] the targets, on [T] which tokens count, ent [T] the targets' sum p log p."""
    loss, lse = fwd()
    dX, dW = bwd(lse)
    assert same_bits((loss, lse), fwd()) and same_bits((dX, dW), bwd(lse))
    X, W, G = X.double() * on[:, None], W.double(), G.double() * on
    z = X @ W.T / temp
    rs = torch.logsumexp(z, 1)
    rl = temp ** 2 * (ent + rs * P.sum(1) - (P * z).sum(1)) * on
    rs = rs * on
    dz = 2.0 ** -17 * (X.abs() @ W.abs().T).max(1).values / temp + 2.0 ** -21
    bounded(lse, rs, on * (dz + 8 * U32 * rs.abs()), "lse")
    bounded(loss, rl, on * temp ** 2 * (2 * dz + 16 * U32 * (rs.abs() + rl.abs() + ent.abs())), "loss")
    q = torch.softmax(z, 1)
    g = (temp * G)[:, None]
    D, A = (q - P) * g, (q + P) * g.abs()
    c, least = U16 + 2.0 ** -12, 2.0 ** -126 * (1 + g.abs())
    for got, ref, mag, floor, what in ((dX, D @ W, A @ W.abs(), least * W.abs().sum(0), "dX"),
                                       (dW, D.T @ X, A.T @ X.abs(), (least * X.abs()).sum(0), "dW")):
        bounded(got, ref, c * mag + U16 * ref.abs() * (1 + c) + floor, what)


def check_labels(train, T, d, V, seed=0, ignored=0.3):
    X, W, g = head_inputs(T, d, V, seed=T + d + V + seed)
    labels = labels_for(T, V, g, ignored)
    G = torch.randn(T, generator=g).to(DEV)
    on = ((labels >= 0) & (labels < V)).to(DEV)
    X, W, labels = X.to(DEV), W.to(DEV), labels.to(DEV)
    P = torch.zeros((T, V), dtype=torch.float64, device=DEV)
    P[on] = torch.nn.functional.one_hot(labels[on], V).double()
    check(lambda: train.cross_entropy_forward(X, W, labels),
          lambda lse: train.cross_entropy_backward(G, X, W, labels, lse), X, W, P, on,
          torch.zeros(T, dtype=torch.float64, device=DEV), 1.0, G)


def check_teacher(train, T, d, V, K, temp):
    X, W, g = head_inputs(T, d, V, seed=T + d + V + K)
    teacher, ids, targets = distill_targets(T, V, K, g, temp)
    P, on, ent = (torch.from_numpy(t).to(DEV) for t in targets)
    G = torch.randn(T, generator=g).to(DEV)
    X, W, teacher, ids = X.to(DEV), W.to(DEV), teacher.to(DEV), ids.to(DEV)
    check(lambda: train.distill_forward(X, W, teacher, ids, temp),
          lambda lse: train.distill_backward(G, X, W, teacher, ids, lse, temp), X, W, P, on, ent, temp, G)


# one tile per pair; several, of widths with one part of a logit and with more
PAIRS = [(300, 1032, 1000, 1), (1100, 968, 9001, 2), (2100, 1032, 5003, 2), (1100, 2056, 9001, 2)]


@pytest.mark.parametrize("T,d,V,tiles", PAIRS)
def test_pairs(train, T, d, V, tiles):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for K in (0, 7):
        for backward in (False, True):
            info = train.head_info(T, V, d, K, backward)
            assert info["logits_ctas"] == 2 and not (backward and info["dX_ctas"] != 2), info
        assert -(-T // 256) * -(-V // 256) > (tiles - 1) * (sms // 2)
    check_labels(train, T, d, V)
    check_teacher(train, T, d, V, 7, 2.0)


@pytest.mark.parametrize("T", [5, 40])
@pytest.mark.parametrize("d", [264, 1032])
@pytest.mark.parametrize("V,columns", [(12001, 128), (20011, 192)])
def test_tiles_of_few_tokens(train, T, d, V, columns):
    """Half of a 192-column tile starts inside a block of the table that finds a row's first entry."""
    for backward in (False, True):
        assert train.head_info(T, V, d, 0, backward)["logits_columns"] == columns
    check_labels(train, T, d, V)
    check_teacher(train, T, d, V, 300, 1.0)


def test_default_pieces(train):
    """The cut that a call without `piece` makes: 8192 columns or more at a time, here two pieces."""
    T, d, V = 20000, 64, 9000
    assert train.head_info(T, V, d, 0, True)["pieces"] == 2
    check_labels(train, T, d, V)


def test_expired_wait_of_a_pair(train):
    """As for single CTAs: no loads are issued, every wait runs out, the status says so, nothing stays behind."""
    from mixture_experts_layer_19_gb300 import moe
    T, d, V = 300, 1032, 777
    assert train.head_info(T, V, d)["logits_ctas"] == 2 and train.head_info(T, V, d, 0, True)["dX_ctas"] == 2
    X, W, g = head_inputs(T, d, V, seed=14)
    X, W, lab, dl = X.to(DEV), W.to(DEV), torch.randint(0, V, (T,), generator=g).to(DEV), torch.ones(T, device=DEV)
    loss, lse = train.cross_entropy_forward(X, W, lab)
    grads = train.cross_entropy_backward(dl, X, W, lab, lse)
    stalled = dict(wait_timeout_ns=20_000_000, debug_flags=train.MOE_DEBUG_STALL_TEST)
    train.cross_entropy_forward(X, W, lab, **stalled)
    assert train.device_status(0) == moe.MOE_ERR_TIMEOUT
    train.cross_entropy_backward(dl, X, W, lab, lse, **stalled)
    assert train.device_status(0) == moe.MOE_ERR_TIMEOUT
    assert train.device_status(0) == 0
    assert same_bits((loss, lse), train.cross_entropy_forward(X, W, lab))
    assert same_bits(grads, train.cross_entropy_backward(dl, X, W, lab, lse))


@pytest.mark.parametrize("T,d,V,K", [(40, 264, 20011, 0), (300, 1032, 1000, 7), (4096, 256, 40000, 0), (20000, 64, 9000, 5),
                                     (131072, 512, 32768, 0), (1 << 20, 64, 100000, 0)])
def test_workspace_is_what_the_header_says(train, T, d, V, K):
    Tp = -(-T // 256) * 256
    forward, backward = (train.head_info(T, V, d, K, b) for b in (False, True))
    common = Tp * (2 * d + 64) + K * Tp * 8 + (Tp * V / 64 + Tp * 4 if K else 0) + 65536
    part = 16 * Tp * (V // forward["logits_columns"] + 1) + 4 * Tp * max(K, 1)
    assert train._head_workspace_bytes(T, V, d, K, 0, False, 0) <= common + part
    piece = max(256 << 20, 16384 * Tp) + 512 * Tp                       # pieces are multiples of 256 columns
    sums = 4 * d * Tp * backward["dX_splits"] if backward["dX_splits"] > 1 or backward["pieces"] > 1 else 0
    got = train._head_workspace_bytes(T, V, d, K, 0, True, 0)
    assert got <= common + min(piece, 2 * Tp * (V + 256)) + sums
    assert got >= min(piece / 2, 2 * Tp * V) + sums                      # and not far below: pieces of equal size
