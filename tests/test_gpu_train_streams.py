"""GPU tests of the training operators on a stream other than their tensors'."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


def calls(train):
    """Name, input maker and call(inputs, stream) of every function that takes a stream."""
    T, d, V, K = 300, 512, 1000, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)                                  # noqa: E731
    X, W, w, b = rand(T, d).to(torch.bfloat16), (rand(V, d) / d ** 0.5).to(torch.bfloat16), rand(d), rand(d)
    lab, ids = (torch.randint(0, V, s, generator=g, device=DEV) for s in ((T,), (T, K)))
    u, dl, dy = rand(T, K), rand(T), rand(T, d).to(torch.bfloat16)
    _, mean, rstd = train.layer_norm_forward(X, w, b)
    lse, lse2 = train.cross_entropy_forward(X, W, lab)[1], train.distill_forward(X, W, u, ids, 2.0)[1]
    return [("layer_norm_forward", (X, w, b), lambda i, s: train.layer_norm_forward(*i, stream=s)),
            ("layer_norm_backward", (dy, X, w, mean, rstd), lambda i, s: train.layer_norm_backward(*i, stream=s)),
            ("cross_entropy_forward", (X, W, lab), lambda i, s: train.cross_entropy_forward(*i, stream=s)),
            ("cross_entropy_backward", (dl, X, W, lab, lse), lambda i, s: train.cross_entropy_backward(*i, stream=s)),
            ("distill_forward", (X, W, u, ids), lambda i, s: train.distill_forward(*i, 2.0, stream=s)),
            ("distill_backward", (dl, X, W, u, ids, lse2), lambda i, s: train.distill_backward(*i, 2.0, stream=s))]


def test_inputs_may_be_dropped_right_after_the_call(train):
    """The side stream is kept busy while the caller drops the inputs and its allocator hands their sizes
    out again: what is written there must not reach the call."""
    side = torch.cuda.Stream()
    for name, inputs, call in calls(train):
        ref = call(inputs, None)
        mine = [t.clone() for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)                                  # about 20 ms
        out = call(mine, side)
        sizes = [(t.shape, t.dtype) for t in mine]
        del mine
        junk = [torch.full(s, 1, dtype=dt, device=DEV) for s, dt in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), name
        del junk


def test_a_stream_of_another_gpu_is_refused(train):
    class Elsewhere:
        device_index = 1

    for name, inputs, call in calls(train):
        with pytest.raises(ValueError, match="stream"):
            call(inputs, Elsewhere())
