"""A layer of experts trained in 8-bit floating point: every expert is an MLP of
its own for the tokens that are routed to it,

    y[t] = x[t] + W2[e] gelu(W1[e] x[t] + b1[e]) + b2[e],   e = expert of t

Activations, gradients and weights enter the products as e4m3 codes with a
power-of-two step per 128 values, products are grouped by expert, the flat
gradient is sent as INT8 with error feedback, clipped, and applied by AdamW whose
states are kept in 8 bits.

    python examples/experts_step.py [--tokens 4096] [--features 1024] [--hidden 2048] [--experts 8] [--steps 20]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from communication_efficient_gradient_amd import gq  # noqa: E402


class Experts:
    """Parameters are slices of one flat fp32 vector, gradients of another."""

    def __init__(self, tokens: int, features: int, hidden: int, experts: int,
                 dtype: torch.dtype = torch.bfloat16, seed: int = 0):
        self.t, self.f, self.h, self.k, self.dtype = tokens, features, hidden, experts, dtype
        shapes = {"w1": (experts, hidden, features), "b1": (experts, hidden),
                  "w2": (experts, features, hidden), "b2": (experts, features)}
        ends = [0]
        for s in shapes.values():
            ends.append(ends[-1] + math.prod(s))
        self.flat, self.grad = (torch.zeros(ends[-1], device="cuda") for _ in range(2))
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.p, self.g = {}, {}
        for (name, s), lo, hi in zip(shapes.items(), ends, ends[1:]):
            self.p[name], self.g[name] = self.flat[lo:hi].view(s), self.grad[lo:hi].view(s)
            if name.startswith("w"):
                self.p[name].normal_(std=s[-1] ** -0.5, generator=gen)
        self.layers = torch.tensor(ends, device="cuda")
        self.decay = torch.tensor([0.01 if n.startswith("w") else 0.0 for n in shapes],
                                  device="cuda")
        # forms: activations of both widths, weights as they lie (forward) and
        # transposed (the input's gradient)
        self.a_f, self.a_h = (gq.act(tokens, c, dtype, 128) for c in (features, hidden))
        self.x8, self.dz8 = gq.alloc_block(self.a_f), gq.alloc_block(self.a_f)
        self.v8, self.du8 = gq.alloc_block(self.a_h), gq.alloc_block(self.a_h)
        self.a_w1 = gq.act(hidden, features, torch.float32, 128)
        self.a_w2 = gq.act(features, hidden, torch.float32, 128)
        self.w1, self.w1t, self.w2, self.w2t = (
            gq.alloc_block_weight(a, experts, transposed=t)
            for a in (self.a_w1, self.a_w2) for t in (False, True))
        n = self.flat.numel()
        self.ws = gq.alloc_workspace(max(
            gq.gq_block_linear_workspace(self.a_f, hidden, experts),
            gq.gq_block_linear_workspace(self.a_h, features, experts),
            gq.gq_block_wgrad_workspace(self.a_f, hidden, experts),
            gq.gq_block_wgrad_workspace(self.a_h, features, experts),
            gq.gq_grad_norm_workspace(n)))
        self.norm, self.scale = (torch.empty(1, device="cuda") for _ in range(2))
        self.pack_weights()

    def new(self, cols: int) -> torch.Tensor:
        return torch.empty(self.t, cols, dtype=self.dtype, device="cuda")

    def pack_weights(self) -> None:
        gq.gq_block_pack_weight(self.a_w1, self.p["w1"], self.w1, self.w1t)
        gq.gq_block_pack_weight(self.a_w2, self.p["w2"], self.w2, self.w2t)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        """x: tokens sorted by expert, offsets: where each expert's begin."""
        self.offsets = offsets
        self.u, z = self.new(self.h), self.new(self.f)
        gq.gq_block_pack(self.a_f, x, *self.x8)
        gq.gq_block_linear(self.a_f, *self.x8, *self.w1, self.p["b1"], self.u,
                           offsets=offsets, workspace=self.ws)
        gq.gq_block_pack(self.a_h, torch.nn.functional.gelu(self.u), *self.v8)
        gq.gq_block_linear(self.a_h, *self.v8, *self.w2, self.p["b2"], z,
                           offsets=offsets, workspace=self.ws)
        return x + z

    def backward(self, dy: torch.Tensor, beta: float = 0.0) -> torch.Tensor:
        """Gradients into self.grad (beta = 1 adds to what is there); returns
        the input's gradient."""
        g, at = self.g, dict(offsets=self.offsets, workspace=self.ws)
        gq.gq_block_wgrad(self.a_h, dy, *self.v8, g["w2"], g["b2"], beta=beta, **at)
        gq.gq_block_pack(self.a_f, dy, *self.dz8)
        dv = self.new(self.h)
        gq.gq_block_linear(self.a_f, *self.dz8, *self.w2t, None, dv, **at)
        du = torch.ops.aten.gelu_backward(dv, self.u)
        gq.gq_block_wgrad(self.a_f, du, *self.x8, g["w1"], g["b1"], beta=beta, **at)
        gq.gq_block_pack(self.a_h, du, *self.du8)
        dx = self.new(self.f)
        gq.gq_block_linear(self.a_h, *self.du8, *self.w1t, None, dx, **at)
        return dx + dy


class Trainer:
    """Sends the gradient as INT8 with error feedback and applies what comes
    back: clipped, AdamW with states in 8 bits."""

    # Both draw random words by element and step, so each has a key of its own
    # (of several workers each sends with another one, and all update with one).
    UPDATE_SEED, SEND_SEED = 0, 1

    def __init__(self, block: Experts, lr: float, max_norm: float = 1.0, bits: int = 8):
        n = block.flat.numel()
        self.block, self.max_norm = block, max_norm
        self.d = gq.desc(gq.GQ_UNIFORM, bucket=512, s=127)
        self.codes, self.meta = gq.alloc_payload(self.d, n)
        self.e, self.mean = (torch.zeros(n, device="cuda") for _ in range(2))
        self.adamw = gq.adamw(lr, bits=bits)
        self.m, self.v = gq.alloc_adamw(self.adamw, n)
        self.step = 0

    def update(self) -> None:
        b, n = self.block, self.block.flat.numel()
        self.step += 1
        gq.gq_quantize(self.d, b.grad, self.e, self.SEND_SEED, self.step, self.codes,
                       self.meta)
        gq.gq_dequantize_accumulate(self.d, n, [self.codes], [self.meta], 1.0, 0.0, self.mean)
        gq.gq_grad_norm(self.mean, self.max_norm, b.norm, b.scale, workspace=b.ws)
        gq.gq_adamw(self.adamw, self.mean, b.flat, self.m, self.v, self.step, b.layers,
                    decay=b.decay, grad_scale=b.scale, seed=self.UPDATE_SEED)
        b.pack_weights()


def routed(tokens: int, experts: int, seed: int = 1) -> torch.Tensor:
    """Offsets of tokens that a router spread unevenly."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    load = torch.softmax(torch.randn(experts, generator=gen, device="cuda"), 0)
    first = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    first[1:] = torch.round(torch.cumsum(load, 0) * tokens).long()
    first[-1] = tokens
    return first


def train(tokens: int, features: int, hidden: int, experts: int, steps: int, say=print):
    """Fits the experts to a fixed random target; returns the losses."""
    block = Experts(tokens, features, hidden, experts)
    trainer = Trainer(block, lr=1e-3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, features, generator=gen, device="cuda").to(block.dtype)
    mix = torch.randn(features, features, generator=gen, device="cuda") * features ** -0.5
    target = x + torch.tanh(x.float() @ mix).to(block.dtype)
    offsets = routed(tokens, experts)
    losses = []
    for step in range(steps):
        diff = block.forward(x, offsets).float() - target.float()
        losses.append(float(diff.square().mean()))
        block.backward((diff * (2.0 / tokens)).to(block.dtype))
        trainer.update()
        say(f"step {step}: loss {losses[-1]:.5f}, gradient's norm {float(block.norm):.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--features", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    if not torch.cuda.is_available():
        sys.exit("experts_step.py needs a GPU")
    train(args.tokens, args.features, args.hidden, args.experts, args.steps)
