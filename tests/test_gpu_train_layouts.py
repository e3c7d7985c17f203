"""GPU tests of what the differentiable training operators take: gradients and inputs that start anywhere.
A layout changes no bit of a result, so every comparison is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def shifted(t, by=1):
    """The same values `by` elements further on in memory."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm_gradient_that_starts_anywhere(train, dtype):
    """cat hands each part a view of its own gradient: at an odd width the second starts off 16 bytes."""
    d, rows = 1001, (3, 5)
    g = gen(1)
    w, b = torch.randn(d, generator=g, device=DEV), torch.randn(d, generator=g, device=DEV)
    xs = [torch.randn((r, d), generator=g, device=DEV).to(dtype).requires_grad_() for r in rows]
    dy = torch.randn((sum(rows), d), generator=g, device=DEV).to(dtype)
    ws, bs = ([t.clone().requires_grad_() for _ in rows] for t in (w, b))
    torch.cat([train.layer_norm(x, wi, bi) for x, wi, bi in zip(xs, ws, bs)]).backward(dy)
    for x, wi, bi, part in zip(xs, ws, bs, dy.split(rows)):
        y, mean, rstd = train.layer_norm_forward(x.detach(), w, b)
        assert equal((x.grad, wi.grad, bi.grad), train.layer_norm_backward(part.clone(), x.detach(), w, mean, rstd))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm_inputs_that_start_anywhere(train, dtype):
    d = 1001
    g = gen(2)
    x = torch.randn((7, d), generator=g, device=DEV).to(dtype)
    w, b = torch.randn(d, generator=g, device=DEV), torch.randn(d, generator=g, device=DEV)
    full = train.layer_norm(x, w, b)
    assert torch.equal(train.layer_norm(x[1:], w, b), full[1:])
    assert torch.equal(train.layer_norm(x, shifted(w), shifted(b)), full)
    assert torch.equal(train.layer_norm(x[:, 1:], w[1:], b[1:]),
                       train.layer_norm(x[:, 1:].contiguous(), w[1:].clone(), b[1:].clone()))


def test_head_activations_that_start_anywhere(train):
    T, d, V = 20, 72, 300
    g = gen(3)
    X = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device=DEV).to(torch.bfloat16)
    lab = torch.randint(0, V, (T,), generator=g, device=DEV)
    u, ids = torch.randn((T, 3), generator=g, device=DEV), torch.randint(0, V, (T, 3), generator=g, device=DEV)
    for call in (lambda x: train.linear_cross_entropy(x, W, lab), lambda x: train.linear_distillation(x, W, u, ids, 2.0)):
        ref = X.clone().requires_grad_()
        call(ref).sum().backward()
        got = shifted(X).requires_grad_()
        assert torch.equal(call(got), call(ref))
        call(got).sum().backward()
        assert torch.equal(got.grad, ref.grad)


def test_strided_targets(train):
    """Labels, teacher logits and ids as columns, transposes and reversed views of larger tensors."""
    T, d, V, K = 40, 64, 300, 4
    g = gen(4)
    X = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device=DEV).to(torch.bfloat16)
    batch = torch.randint(0, V, (T, 2), generator=g, device=DEV)
    u, ids = torch.randn((K, T), generator=g, device=DEV), torch.randint(0, V, (T, 2 * K), generator=g, device=DEV)
    for call, targets in ((train.linear_cross_entropy, (batch[:, 1],)),
                          (train.linear_distillation, (u.t(), ids[:, ::2]))):
        grads = []
        for ts in (targets, [t.contiguous() for t in targets]):
            x, w = X.clone().requires_grad_(), W.clone().requires_grad_()
            loss = call(x, w, *ts)
            loss.sum().backward()
            grads.append((loss, x.grad, w.grad))
        assert equal(*grads)


@pytest.mark.parametrize("lead", [(), (3,), (2, 5), (2, 0), (2, 3, 4)])
def test_head_of_a_leading_shape(train, lead):
    """The head takes [..., d], as the norm does, and gives a loss of that leading shape."""
    d, V, K = 64, 300, 4
    g = gen(5)
    X = torch.randn((*lead, d), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device=DEV).to(torch.bfloat16)
    lab, ids = (torch.randint(0, V, s, generator=g, device=DEV) for s in (lead, (*lead, K)))
    u = torch.randn((*lead, K), generator=g, device=DEV)
    T = lab.numel()
    for call, targets in ((train.linear_cross_entropy, (lab,)), (train.linear_distillation, (u, ids))):
        x, x2 = X.clone().requires_grad_(), X.reshape(T, d).clone().requires_grad_()
        loss = call(x, W, *targets)
        flat = call(x2, W, *[t.reshape(T, *t.shape[len(lead):]) for t in targets])
        assert loss.shape == lead and torch.equal(loss.reshape(T), flat)
        loss.sum().backward()
        flat.sum().backward()
        assert torch.equal(x.grad.reshape(T, d), x2.grad)
    x = torch.zeros((2, 3, d), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: train.linear_cross_entropy(x, W, torch.zeros(6, dtype=torch.int64, device=DEV)),
                 lambda: train.linear_distillation(x, W, torch.zeros((2, 4, K), device=DEV),
                                                   torch.zeros((2, 4, K), dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            call()
