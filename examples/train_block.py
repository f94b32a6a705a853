"""Train one residual MLP block whose two layers are residual-binarized, on synthetic data.

One step, all of it in the library's kernels but for the loss and the clip factor:

  derive      What_up, What_down from the shared fp32 weights and their scales      qat_derive
  forward     S0 = embedding, X0 = norm(S0)                                        resnorm_forward
              H = silu(X0 What_up^T + b)                                           qat_linear
              O = H What_down^T                                                    qat_linear
              S1 = S0 + gate * norm(O), X1 = norm(S1)                              resnorm_forward
  backward    the same in reverse          resnorm_backward, qat_backward, qat_linear_backward
  update      weights, scales, norms, gate and bias at once                        adamw_step

Usage: python examples/train_block.py [--tokens 512] [--width 1024] [--hidden 2752] [--planes 2]
                                      [--steps 40] [--bits 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import residual_binarized_weight_amd as rb  # noqa: E402


class Layer:
    """A coupled-training layer: the shared weight, its scales, and buffers for what is derived of them."""

    def __init__(self, n_out: int, n_in: int, planes: int, gen: torch.Generator):
        self.W = torch.randn((n_out, n_in), generator=gen, device="cuda") * n_in ** -0.5
        # paths of magnitude |W|, |W| / 2, ... near the mean of |W|
        self.g = torch.stack([self.W.abs().mean(1) * 0.5 ** i for i in range(planes)])
        self.h = torch.ones((planes, n_in), device="cuda")
        self.planes = torch.zeros((planes, n_out, (n_in + 31) // 32), dtype=torch.int32, device="cuda")
        self.What = torch.empty((n_out, n_in), dtype=torch.bfloat16, device="cuda")
        self.dW, self.dg, self.dh = (torch.zeros_like(t) for t in (self.W, self.g, self.h))

    def derive(self):
        rb.qat_derive(self.W, self.g, self.h, planes=self.planes, What=self.What)

    def backward(self, dY, X):
        """dX; the layer's own gradients into its buffers."""
        return rb.qat_backward(dY, X, self.What, self.planes, self.g, self.h, dW=self.dW, dg=self.dg, dh=self.dh)[1]


class Block:
    def __init__(self, width: int, hidden: int, planes: int = 2, bits: int = 32, seed: int = 0, lr: float = 2e-3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.up, self.down = Layer(hidden, width, planes, gen), Layer(width, hidden, planes, gen)
        one = lambda: torch.ones(width, device="cuda")  # noqa: E731
        self.vec = {"w_in": one(), "w_post": one(), "w_out": one(), "gate": one() * 0.5,
                    "bias": torch.zeros(hidden, device="cuda")}
        self.dvec = {k: torch.zeros_like(v) for k, v in self.vec.items()}
        self.weights, self.dweights = [self.up.W, self.down.W], [self.up.dW, self.down.dW]
        small = [self.up.g, self.up.h, self.down.g, self.down.h, *self.vec.values()]
        dsmall = [self.up.dg, self.up.dh, self.down.dg, self.down.dh, *self.dvec.values()]
        self.params, self.grads = self.weights + small, self.dweights + dsmall
        # only the weights decay
        self.plan = rb.adamw_plan(self.params, self.grads, state_bits=bits,
                                  weight_decay=[0.01] * len(self.weights) + [0.0] * len(small))
        self.lr, self.steps = lr, 0

    def forward(self, emb):
        """X1 [M][width] of the embedding (bf16); keeps what the backward needs."""
        v = self.vec
        self.up.derive()
        self.down.derive()
        self.emb = emb
        self.S0 = torch.empty(emb.shape, device="cuda")
        _, self.X0, self.st0 = rb.resnorm_forward(emb, None, v["w_in"], S=self.S0)
        self.H, self.Z = rb.qat_linear(self.X0, self.up.What, bias=v["bias"], act="silu", save_z=True)
        self.O, _ = rb.qat_linear(self.H, self.down.What)
        self.S1, X1, self.st1 = rb.resnorm_forward(self.O, self.S0, v["w_out"], w_post=v["w_post"], gate=v["gate"])
        return X1

    def backward(self, dX1):
        v, d = self.vec, self.dvec
        r = rb.resnorm_backward(dX1, None, self.O, self.S1, self.st1, v["w_out"], w_post=v["w_post"], gate=v["gate"],
                                out={"dw_pre": d["w_out"], "dw_post": d["w_post"], "dgate": d["gate"]})
        dH = self.down.backward(r["dY"], self.H)
        dZ, _ = rb.qat_linear_backward(dH, self.Z, act="silu", db=d["bias"])
        dX0 = self.up.backward(dZ, self.X0)
        return rb.resnorm_backward(dX0, r["dR"], self.emb, self.S0, self.st0, v["w_in"], out={"dw_pre": d["w_in"]})["dY"]

    def update(self, clip: float = 1.0):
        """One optimizer step; the clip factor stays on the device, a step with a bad gradient is skipped."""
        norm = torch.stack(torch._foreach_norm(self.grads)).norm()
        skip = torch.isfinite(norm).logical_not().to(torch.int32)
        scale = (clip / norm).clamp(max=1.0)
        self.steps += 1
        rb.adamw_step(self.plan, self.steps, self.lr, beta2=0.99, grad_scale=scale, skip=skip, seed=1)


def train(tokens=512, width=1024, hidden=2752, planes=2, steps=40, bits=32, seed=0, verbose=False):
    """Losses of the steps: the block learns X1 = norm(x A) of a fixed random rotation-like A."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    A = torch.randn((width, width), generator=gen, device="cuda") * width ** -0.5
    block, losses = Block(width, hidden, planes, bits, seed), []
    emb = torch.randn((tokens, width), generator=gen, device="cuda").to(torch.bfloat16)
    want = emb.float() @ A
    for step in range(steps):
        X1 = block.forward(emb)
        err = X1.float() - want
        losses.append(err.square().mean())
        block.backward((err * (2.0 / err.numel() * tokens)).to(torch.bfloat16))
        block.update()
        if verbose and (step % 10 == 0 or step == steps - 1):
            print(f"step {step:4d}  loss {losses[-1].item():.4f}", flush=True)
    return [float(x) for x in torch.stack(losses).cpu()]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 1024), ("hidden", 2752), ("planes", 2), ("steps", 40), ("bits", 8)):
        ap.add_argument(f"--{name}", type=int, default=default)
    train(**vars(ap.parse_args()), verbose=True)


if __name__ == "__main__":
    main()
