"""GPU tests of NVFP4 weights quantised with tensor scales that the caller gives.

Weights that are cut off at one value lie on borders between codes by the thousand, so that a scale one place off makes
another layer of them: 8 % of the outputs here, by the fp64 oracle.  Kernels are held to what the layer for few
tokens is held to (test_gpu_few.py): 2^-8 for the rounding and 2e-2 for codes of h."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300 import moe
from mixture_experts_layer_19_gb300.workload import to_f64
from oracle import moe_ref, nvfp4
from tests.util import cpu_and_gpu_inputs, rel_err_norm

pytestmark = pytest.mark.gpu


def test_given_scales_decide_the_codes():
    T, d, F, E, k = 24, 1024, 512, 8, 2
    g, h = cpu_and_gpu_inputs(T, d, F, E, k, seed=3)
    for n in ("Wg", "Wu", "Wd"):
        g[n] = g[n].clamp(-0.0645, 0.0645)
        h[n] = to_f64(g[n])
    W = (g["Wg"], g["Wu"], g["Wd"])
    own = nvfp4.weight_scales(h["Wg"], h["Wu"], h["Wd"])
    beside = tuple(np.nextafter(s, np.float32(1), dtype=np.float32) for s in own)

    def oracle(scales):
        return moe_ref.forward(h["X"], h["logits"], h["Wg"], h["Wu"], h["Wd"], k, mx="nvfp4", wscales=scales)[0]
    refs = [oracle(own), oracle(beside)]
    assert rel_err_norm(refs[1], refs[0]) > 5e-2
    with moe.Plan(moe.Config(T_max=T, d=d, F=F, E=E, k=k, prec=moe.MOE_NVFP4)) as plan:
        outs = []
        for scales in (None, beside, own):
            given = None if scales is None else torch.tensor(np.array(scales), device="cuda")
            plan.quantize_weights(*W, scales=given)
            assert plan.nv_weight_scales().tolist() == [float(s) for s in (scales or own)]
            ref = refs[1] if scales is beside else refs[0]
            outs.append(plan.forward_few(g["X"], g["logits"], *W))
            assert rel_err_norm(outs[-1], ref) <= 2.0 ** -8 + 2e-2
            Y, saved = plan.forward(g["X"], g["logits"], *W)
            assert rel_err_norm(Y, ref) <= 4e-2
            plan.backward(g["dY"], g["X"], *W, saved)
        assert torch.equal(outs[0], outs[2])             # the scales it takes itself, handed over
        assert plan.device_status() == 0


def test_refusals():
    g, _ = cpu_and_gpu_inputs(4, 256, 256, 4, 2)
    W = (g["Wg"], g["Wu"], g["Wd"])
    one = torch.ones(2, device="cuda")
    for prec in (moe.MOE_BF16, moe.MOE_MXFP8, moe.MOE_NVFP4):
        with moe.Plan(moe.Config(T_max=4, d=256, F=256, E=4, k=2, prec=prec)) as plan:
            for bad in (one.double(), one[:1], one.cpu(), torch.ones((2, 2), device="cuda")[:, 0]):
                with pytest.raises(ValueError):
                    plan.quantize_weights(*W, scales=bad)
            if prec == moe.MOE_NVFP4:
                plan.quantize_weights(*W, scales=one)
            else:
                with pytest.raises(moe.MoEError):
                    plan.quantize_weights(*W, scales=one)
