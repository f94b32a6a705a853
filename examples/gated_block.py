"""Train one residual gated MLP block whose three layers are residual-binarized, then decode with it in 4 bits.

One step, all of it in the library's kernels but for the loss and the clip factor:

  derive      What_gate, What_up, What_down from the shared fp32 weights and their scales      qat_derive
  forward     S0 = embedding, X0 = norm(S0)                                        resnorm_forward
              H = silu(X0 What_gate^T) (X0 What_up^T)                              qat_glu
              O = H What_down^T                                                    qat_linear
              S1 = S0 + norm(O), X1 = norm(S1)                                     resnorm_forward
  backward    the same in reverse          resnorm_backward, qat_backward, qat_glu_backward, qat_glu_dx
  update      the three weights            muon_step;  scales and norms at once    adamw_step
  decode      the effective weights, which the block was trained through, in 4 bits   q4_pack, q4_glu, q4_gemv

Usage: python examples/gated_block.py [--tokens 512] [--width 1024] [--hidden 2752] [--planes 2] [--steps 40]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import residual_binarized_weight_amd as rb  # noqa: E402
from examples.train_block import Layer  # noqa: E402


class GatedBlock:
    def __init__(self, width: int, hidden: int, planes: int = 2, seed: int = 0, lr: float = 2e-3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gate, self.up, self.down = (Layer(*s, planes, gen) for s in ((hidden, width), (hidden, width), (width, hidden)))
        self.layers = [self.gate, self.up, self.down]
        self.vec = {k: torch.ones(width, device="cuda") for k in ("w_in", "w_post", "w_out")}
        self.dvec = {k: torch.zeros_like(v) for k, v in self.vec.items()}
        self.mom = [torch.zeros_like(y.W) for y in self.layers]
        self.small = [t for y in self.layers for t in (y.g, y.h)] + list(self.vec.values())
        self.dsmall = [t for y in self.layers for t in (y.dg, y.dh)] + list(self.dvec.values())
        self.plan = rb.adamw_plan(self.small, self.dsmall)
        self.lr, self.steps = lr, 0

    def forward(self, emb):
        """X1 [M][width] of the embedding (bf16); keeps what the backward needs."""
        v = self.vec
        for y in self.layers:
            y.derive()
        self.emb = emb
        self.S0 = torch.empty(emb.shape, device="cuda")
        _, self.X0, self.st0 = rb.resnorm_forward(emb, None, v["w_in"], S=self.S0)
        self.H, self.G, self.U = rb.qat_glu(self.X0, self.gate.What, self.up.What, act="silu", save=True)
        self.O, _ = rb.qat_linear(self.H, self.down.What)
        self.S1, X1, self.st1 = rb.resnorm_forward(self.O, self.S0, v["w_out"], w_post=v["w_post"])
        return X1

    def backward(self, dX1):
        v, d = self.vec, self.dvec
        r = rb.resnorm_backward(dX1, None, self.O, self.S1, self.st1, v["w_out"], w_post=v["w_post"],
                                out={"dw_pre": d["w_out"], "dw_post": d["w_post"]})
        dH = self.down.backward(r["dY"], self.H)
        dG, dU, _, _ = rb.qat_glu_backward(dH, self.G, self.U, act="silu")
        for y, dY in ((self.gate, dG), (self.up, dU)):
            rb.qat_backward(dY, self.X0, y.What, y.planes, y.g, y.h, dW=y.dW, dg=y.dg, dh=y.dh, need_dx=False)
        dX0 = rb.qat_glu_dx(dG, dU, self.gate.What, self.up.What)
        return rb.resnorm_backward(dX0, r["dR"], self.emb, self.S0, self.st0, v["w_in"], out={"dw_pre": d["w_in"]})["dY"]

    def update(self, clip: float = 1.0):
        """One optimizer step; the clip factor stays on the device, a step with a bad gradient is skipped."""
        norm = torch.stack(torch._foreach_norm([y.dW for y in self.layers] + self.dsmall)).norm()
        skip = torch.isfinite(norm).logical_not().to(torch.int32)
        scale = (clip / norm).clamp(max=1.0)
        self.steps += 1
        for y, m in zip(self.layers, self.mom):
            rb.muon_step(y.W, y.dW, m, self.lr, weight_decay=0.01, grad_scale=scale, skip=skip)
        rb.adamw_step(self.plan, self.steps, self.lr, beta2=0.99, grad_scale=scale, skip=skip)

    def pack(self, group: int = 64):
        """The weights that the forward multiplies by, in 4 bits, for decode: those of the shared weights and scales
        as they are now."""
        for y in self.layers:
            y.derive()
        self.packed = [rb.q4_pack(y.What, group=group) for y in self.layers]
        self.group = group

    def decode(self, emb):
        """X1 [M][width] of up to 16 tokens' embeddings (bf16) on the packed weights."""
        v, (gate, up, down) = self.vec, self.packed
        S0, X0, _ = rb.resnorm_forward(emb, None, v["w_in"], S=torch.empty(emb.shape, device="cuda"))
        H = rb.q4_glu(gate, up, X0, self.gate.W.shape[0], group=self.group, act="silu")
        O = rb.q4_gemv(*down, H, self.down.W.shape[0], group=self.group)
        return rb.resnorm_forward(O, S0, v["w_out"], w_post=v["w_post"])[1]


def train(tokens=512, width=1024, hidden=2752, planes=2, steps=40, seed=0, verbose=False):
    """(losses, block): the block learns X1 = norm(x A) of a fixed random rotation-like A."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    A = torch.randn((width, width), generator=gen, device="cuda") * width ** -0.5
    block, losses = GatedBlock(width, hidden, planes, seed), []
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
    return [float(x) for x in torch.stack(losses).cpu()], block


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 1024), ("hidden", 2752), ("planes", 2), ("steps", 40)):
        ap.add_argument(f"--{name}", type=int, default=default)
    _, block = train(**vars(ap.parse_args()), verbose=True)
    block.pack()
    token = block.emb[:1]
    print("one token in 4 bits:", block.decode(token).float().norm().item(), "binarized:", block.forward(token).float().norm().item())


if __name__ == "__main__":
    main()
