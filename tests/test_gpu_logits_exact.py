"""GPU tests that logits are processed by the operations that include/moe.h states, one at a time in fp32: equal to the
bit to the same operations of numpy, which rounds each of them once, as IEEE 754 has it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def serve():
    from mixture_experts_layer_19_gb300 import serve
    return serve


def stepwise(z, history, lengths, prompt, rep, freq, pres, bias_ids, bias):
    """z [T, V] fp32, in numpy's fp32."""
    z = z.copy()
    f32 = np.float32
    for t in range(z.shape[0]):
        used = history[t, :lengths[t]]
        for v in np.unique(used):
            if not 0 <= v < z.shape[1]:
                continue
            z[t, v] = z[t, v] / rep[t] if z[t, v] > 0 else z[t, v] * rep[t]
            n = int((used[prompt[t]:] == v).sum())
            if n:
                z[t, v] = f32(f32(z[t, v] - f32(freq[t] * f32(n))) - pres[t])
        for v, b in zip(bias_ids[t], bias[t]):
            if 0 <= v < z.shape[1]:
                z[t, v] = f32(z[t, v] + b)
    return z


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,L,K", [(1, 300, 70, 40), (6, 4099, 900, 1024), (40, 9001, 300, 33), (3, 70000, 5000, 64)])
def test_every_operation_rounds_once(serve, T, V, L, K, dtype):
    g = torch.Generator().manual_seed(V)
    z = (3 * torch.randn((T, V), generator=g)).to(dtype)
    few = torch.randint(0, 40, (T, L), generator=g)
    history = torch.where(torch.rand((T, L), generator=g) < 0.5, torch.randint(-2, V + 2, (T, L), generator=g), few)
    lengths = torch.randint(1, L + 1, (T,), generator=g).to(torch.int32)
    prompt = (lengths * torch.rand(T, generator=g)).to(torch.int32)
    rep, freq, pres = 0.6 + torch.rand(T, generator=g), torch.rand(T, generator=g), torch.rand(T, generator=g)
    bias_ids = torch.randint(-1, min(V + 1, 3 * K // 2), (T, K), generator=g)       # many ids more than once
    bias = torch.randn((T, K), generator=g) * 10.0 ** torch.randint(-3, 6, (T, K), generator=g)
    args = (history, lengths, prompt, rep, freq, pres, bias_ids, bias)
    ref = stepwise(z.float().numpy(), *(a.numpy() for a in args))
    got = serve.process_logits(z.to(DEV), *(a.to(DEV) for a in args))
    assert torch.equal(got.cpu(), torch.from_numpy(ref).to(dtype))


def test_small_repetitions_and_cancelling_biases(serve):
    z = torch.tensor([[1e-5, -1e-5, 1.0, 5.0, 0.0]], device=DEV)
    h = torch.tensor([[0, 1]], device=DEV)
    out = serve.process_logits(z, h, repetition=torch.tensor([1e-39], device=DEV))     # its reciprocal is infinite
    assert out[0, 0].item() == float(np.float32(1e-5) / np.float32(1e-39)) and np.isfinite(out[0, 0].item())
    assert out[0, 1:].tolist() == [float(np.float32(-1e-5) * np.float32(1e-39)), 1.0, 5.0, 0.0]
    ids = torch.tensor([[2, 3, 2, 2, 9]], device=DEV)
    out = serve.process_logits(z, bias_ids=ids, bias=torch.tensor([[1e8, 2.0, -1e8, 0.5, 7.0]], device=DEV))
    assert out[0, 2:].tolist() == [0.5, 7.0, 0.0]                                       # (1 + 1e8) - 1e8 + 0.5
