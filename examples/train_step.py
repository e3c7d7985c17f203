"""A training step around the MoE layer, with its operators used together:

    h = LayerNorm(x);  y = x + MoE(h);  f = LayerNorm(y)
    cross entropy of f against labels, then distillation from a teacher's top logits

on random data, with plain gradient descent.  Run it on a GB300 after
``python -m mixture_experts_layer_19_gb300.build``:

    python examples/train_step.py --tokens 1024 --width 1024 --vocab 32000
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_19_gb300 import moe, train  # noqa: E402


class Block(torch.nn.Module):
    """One pre-norm MoE block with the loss head behind it."""

    def __init__(self, a):
        super().__init__()
        self.norm_in = train.LayerNorm(a.width)
        self.layer = moe.RoutedMoELayer(a.width, a.ffn, a.experts, a.top_k, a.tokens)
        self.norm_out = train.LayerNorm(a.width)
        self.head = train.LMHead(a.width, a.vocab)

    def features(self, x):
        return self.norm_out(x + self.layer(self.norm_in(x)))


def teacher_top(model, x, k):
    """A teacher's largest logits and their ids (here: another model of the same shape)."""
    with torch.no_grad():
        top = (model.features(x) @ model.head.weight.t()).float().topk(k, dim=1)
    return top.values.contiguous(), top.indices.contiguous()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--ffn", type=int, default=512)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--teacher-k", type=int, default=16)
    p.add_argument("--temperature", type=float, default=2.0)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--lr", type=float, default=0.5)
    a = p.parse_args(argv)

    torch.manual_seed(0)
    x = torch.randn((a.tokens, a.width), device="cuda").to(torch.bfloat16)
    labels = torch.randint(0, a.vocab, (a.tokens,), device="cuda")
    labels[::8] = -100                                   # tokens of the prompt: no loss
    student = Block(a)
    values, ids = teacher_top(Block(a), x, a.teacher_k)
    opt = torch.optim.SGD(student.parameters(), lr=a.lr)
    counted = (labels >= 0).sum()

    losses = {"cross entropy": [], "distillation": []}
    for kind, out in losses.items():
        for _ in range(a.steps):
            f = student.features(x)
            if kind == "cross entropy":
                loss = student.head(f, labels).sum() / counted
            else:
                loss = student.head.distill(f, values, ids, a.temperature).mean()
            opt.zero_grad()
            loss.backward()
            opt.step()
            out.append(float(loss.detach()))
        print(f"{kind}: {out[0]:.4f} -> {out[-1]:.4f} in {a.steps} steps")
    if train.device_status() or student.layer.plan.device_status():
        raise RuntimeError("a device-side wait expired")
    return losses


if __name__ == "__main__":
    main()
