"""A mixture-of-experts layer on mxfp4 experts, and the training of its router.

Forward, per token x [D] (E experts of width F, k a token):
    logits        = x gate^T                                   a plain product
    weights, ids  = moe_route(logits)                          k experts, their weights
    h             = gather_mxfp4_matmul(x, up, ids)            [k, 2 F], gate and up halves
    o             = gather_mxfp4_matmul(h, down, ids, swiglu)  [k, D]
    y             = moe_combine(o, weights)
The experts stay as they are; the router learns from grad_y through
moe_combine_grad (the weights' gradient) and moe_route_grad (the logits'), and
its balance bias moves towards the experts that get fewer tokens.

    python examples/moe_layer.py [--tokens 4096] [--experts 64] [--choice 8] [--dim 2048] [--width 768] [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_matmul_amd as qm  # noqa: E402


class MoELayer:
    """gate [E, D]; up [E, 2 F, D] and down [E, D, F], quantized to mxfp4 here."""

    def __init__(self, gate, up, down, k, score="sigmoid"):
        self.gate = gate.float()
        self.bias = torch.zeros(gate.shape[0], device=gate.device)
        self.up = qm.quantize(up, mode="mxfp4")
        self.down = qm.quantize(down, mode="mxfp4")
        self.k, self.score = k, score

    def forward(self, x):
        """y [T, D] for x [T, D], and what the backward pass needs."""
        logits = x.float() @ self.gate.t()
        weights, ids = qm.moe_route(logits, self.k, score=self.score, bias=self.bias)
        h = qm.gather_mxfp4_matmul(x, self.up, ids)
        o = qm.gather_mxfp4_matmul(h.view(-1, h.shape[-1]), self.down, ids.view(-1), activation="swiglu")
        o = o.view(*ids.shape, -1)
        return qm.moe_combine(o, weights, ids), (x, logits, weights, ids, o)

    def gate_gradient(self, saved, grad_y):
        """Gradient of the gate for grad_y [T, D]; the choice of experts carries none."""
        x, logits, weights, ids, o = saved
        _, grad_weights = qm.moe_combine_grad(grad_y, o, weights, ids)
        grad_logits = qm.moe_route_grad(logits, ids, grad_weights, score=self.score)
        return grad_logits.t() @ x.float()

    def balance(self, ids, rate):
        """Moves the bias of each expert towards the mean load; returns the largest load over the mean."""
        load = torch.bincount(ids[ids >= 0], minlength=self.bias.numel()).float()
        self.bias += rate * torch.sign(load.mean() - load)
        return (load.max() / load.mean()).item()


def random_layer(E, k, D, F, device="cuda", seed=0):
    g = torch.Generator(device).manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()

    return MoELayer(normal(E, D, std=D ** -0.5), normal(E, 2 * F, D, std=D ** -0.5), normal(E, D, F, std=F ** -0.5), k)


def train_router(layer, teacher_gate, tokens, steps, rate=10.0, balance_rate=0.0, seed=1):
    """Fits the layer's gate to outputs of the same experts under teacher_gate; returns each step's relative loss."""
    D, device = layer.gate.shape[1], layer.gate.device
    g = torch.Generator(device).manual_seed(seed)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, D, generator=g, device=device).bfloat16()
        own, layer.gate = layer.gate, teacher_gate
        target = layer.forward(x)[0].float()
        layer.gate = own
        y, saved = layer.forward(x)
        diff = y.float() - target
        scale = target.square().mean()
        losses.append((diff.square().mean() / scale).item())
        grad = layer.gate_gradient(saved, (2 * diff / (scale * D)).to(y.dtype))
        layer.gate = layer.gate - rate * grad / tokens
        if balance_rate:
            layer.balance(saved[3], balance_rate)
    return losses


def time_forward(layer, tokens, passes=20):
    """Microseconds of a forward pass among others."""
    x = torch.randn(tokens, layer.gate.shape[1], device=layer.gate.device).bfloat16()
    for _ in range(3):
        layer.forward(x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(passes):
        layer.forward(x)
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / passes * 1e3


def main(argv=None):
    p = argparse.ArgumentParser(description="A mixture-of-experts layer on mxfp4 experts.")
    for name, value in (("tokens", 4096), ("experts", 64), ("choice", 8), ("dim", 2048), ("width", 768), ("steps", 40)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    layer = random_layer(a.experts, a.choice, a.dim, a.width)
    for tokens in sorted({1, 64, a.tokens}):
        us = time_forward(layer, tokens)
        print(f"forward, {tokens} tokens x {a.choice} of {a.experts} experts: {us:.1f} us", flush=True)
    teacher = layer.gate.clone()
    layer.gate = teacher + 0.5 * teacher.std() * torch.randn_like(teacher)
    losses = train_router(layer, teacher, a.tokens, a.steps)
    print(f"router training: relative loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps", flush=True)
    return losses


if __name__ == "__main__":
    main()
