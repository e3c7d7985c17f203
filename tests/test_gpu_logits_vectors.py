"""GPU test of each instantiation of the logits' kernel: one to eight 16-byte vectors per thread, by the rule that picks as
few as give every SM a block."""
import pytest
import torch

from tests.test_gpu_logits import check, inputs, on

pytestmark = pytest.mark.gpu
V = 9001


def vectors(T, width, sms):
    n = 32 // width
    most = V + width - 1                                 # rows of 9001 do not all start on 16 bytes
    while n > 1 and T * -(-most // (256 * n * width)) < sms:
        n //= 2
    return n


@pytest.mark.parametrize("dtype,width", [(torch.float32, 4), (torch.bfloat16, 8)])
def test_every_number_of_vectors(dtype, width):
    from mixture_experts_layer_19_gb300 import serve
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    first = {}
    for T in range(1, 2 * sms):
        first.setdefault(vectors(T, width, sms), T)
    assert sorted(first) == [n for n in (1, 2, 4, 8) if n <= 32 // width]
    for T in first.values():
        s = inputs(T, V, 30, 5, 2, dtype, seed=T)
        check(serve.process_logits(**on(s)), s)
