"""The layer with FP8 expert weights, as a server and a trainer would run it:

  python examples/fp8_layer.py

Serving: the weights are quantised once; a prompt goes through forward()
(tokens quantised in the dispatch, FP8 expert matmuls), then tokens are decoded
one step at a time from the same weights through forward_few() (two launches a
step).  Training: a grouped projection with its forward, data gradient and
weight gradient in FP8, fitted to another one's outputs by gradient steps on
bf16 weights that are quantised again after each step.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_expert_layer_04_gb300.layer import Dims, GroupedLinearFP8, MoELayer


def randn(gen, std, *shape):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def serve(gen, prompt=512, steps=8, d=1024, E=32, k=4, I=512):
    """Prints how far the FP8 layer is from the bf16 one; returns the two
    relative differences (prompt, decoded tokens)."""
    w = dict(W_g=randn(gen, 1.28 / d ** 0.5, E, d), W13=randn(gen, 1.3 / d ** 0.5, E + 1, 2 * I, d),
             W2=randn(gen, 1.3 / I ** 0.5, E + 1, d, I))
    bias = torch.zeros(2, E, device="cuda")
    dims = Dims(prompt, d, E, k, I)
    fp8, bf16 = (MoELayer(dims, w, scaling=2.5, fp8=f) for f in (True, False))
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())

    x = randn(gen, 1.0, prompt, d)
    first = rel(fp8.forward(x, bias), bf16.forward(x, bias))
    decoded = 0.0
    for _ in range(steps):
        x = randn(gen, 1.0, 1, d)
        decoded = max(decoded, rel(fp8.forward_few(x, bias), bf16.forward_few(x, bias)))
    print(f"serving: FP8 against bf16, relative difference {first:.4f} on the prompt, "
          f"at most {decoded:.4f} on {steps} decoded tokens")
    return first, decoded


def train(gen, steps=30, G=4, rows=512, N=256, K=384):
    """Prints and returns the first and the last loss."""
    target = randn(gen, K ** -0.5, G, N, K)
    weight = randn(gen, K ** -0.5, G, N, K)
    master = weight.float()
    layer = GroupedLinearFP8(weight, rows)
    # uneven groups, one of them empty
    offsets = torch.tensor([0, rows // 2, rows // 2, rows - 37, rows], dtype=torch.int32,
                           device="cuda")
    cut = offsets.tolist()
    losses = []
    for _ in range(steps):
        x = randn(gen, 1.0, rows, K)
        want = torch.cat([x[a:b] @ target[g].T for g, (a, b) in enumerate(zip(cut, cut[1:]))])
        diff = layer.forward(x, offsets).float() - want.float()
        losses.append(float(diff.square().mean()))
        layer.backward(diff.to(torch.bfloat16))
        master -= 1e-3 * layer.dW
        weight.copy_(master)
        layer.quantize_weights()
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    return losses[0], losses[-1]


if __name__ == "__main__":
    g = torch.Generator(device="cuda").manual_seed(0)
    serve(g)
    train(g)
