"""GPU tests of distillation targets at the ends of their types' range, against the fp64 oracle with the
bounds of tests/test_gpu_train.py: a logit divided by the temperature may leave fp32, its distance to the
row's largest one may not."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300.workload import to_f64
from oracle import train_ref
from tests.test_gpu_train import check_head, head_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


@pytest.mark.parametrize("temp", [0.25, 1.0, 2.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [20, 150])
def test_teacher_logits_at_the_ends_of_the_range(train, T, dtype, temp):
    """A mask of the type's lowest value is a logit like any other: alone in a row it is the teacher's
    distribution, beside others it has no weight.  Only -inf takes an entry out."""
    V, K = 400, 5
    X, W, g = head_inputs(T, 64, V, seed=T)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)])
    teacher = torch.randn((T, K), generator=g).to(dtype)
    low, top = torch.finfo(dtype).min, torch.finfo(dtype).max
    teacher[0::5, 1:] = low                                # one logit, the rest masked
    teacher[1::5] = low                                    # nothing but the mask
    teacher[2::5, 2] = top
    teacher[2::5, 3] = low
    teacher[3::5, :3] = -np.inf                            # not in use, the rest masked
    teacher[3::5, 3:] = low
    targets = train_ref.teacher_targets(to_f64(teacher), ids.numpy(), V, temp)
    assert targets[1].all()
    check_head(train, X, W, torch.full((T,), 1.0 / T), targets, temp, teacher=teacher, ids=ids)
