"""The block of examples/gated_block.py, its operators run together: gradients against autograd in 64 bits, the update
against the oracle's, and a decoded token on the packed weights.

The gradients pass through bf16 activations and weights (unit roundoff 2^-8) several times: each tensor's 2-norm
error is bounded by 2^-8 times the number of bf16 roundings on its longest path (at most 9: What, X0, G or U, H, O, dX1, dO,
dH, dG or dU), taken at full size.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import residual_binarized_weight_amd as rb
from oracle import block_oracle as BO

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs the GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rms(x, w):
    return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w


def reference(e, gate, up, down, v):
    """X1 of the block in 64 bits."""
    x0 = rms(e, v["w_in"])
    g = x0 @ gate.t()
    o = (g * torch.sigmoid(g) * (x0 @ up.t())) @ down.t()
    return rms(e + rms(o, v["w_post"]), v["w_out"])


@pytest.mark.parametrize("M,D,Hd", [(96, 200, 344), (37, 75, 130)])
def test_gradients_of_the_block(M, D, Hd):
    torch.manual_seed(0)
    b = example().GatedBlock(D, Hd, planes=2, seed=3)
    for x in b.vec.values():
        x.add_(torch.randn_like(x) * 0.2)
    emb = torch.randn((M, D), device="cuda").to(torch.bfloat16)
    dX1 = torch.randn((M, D), device="cuda").to(torch.bfloat16)
    X1 = b.forward(emb)
    demb = b.backward(dX1)
    torch.cuda.synchronize()
    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    v = {k: leaf(x) for k, x in b.vec.items()}
    w = [leaf(y.What.float()) for y in b.layers]
    e = leaf(emb.float())
    x1 = reference(e, *w, v)
    x1.backward(dX1.double().cpu())
    rel = lambda a, r: float((a.double().cpu() - r).norm() / r.norm())  # noqa: E731
    lim = 9 * 2.0 ** -8
    assert rel(X1.float(), x1.detach()) <= lim
    for got, ref in ((demb.float(), e.grad), *((y.dW, t.grad) for y, t in zip(b.layers, w)), *((b.dvec[k], v[k].grad) for k in v)):
        assert rel(got, ref) <= lim, rel(got, ref)


def test_gradient_of_the_gate_against_differences():
    """The block's own forward, in fp32 outputs, at W and at W + e D along the gradient's direction."""
    torch.manual_seed(1)
    M, N, K = 64, 96, 80
    X, Wg, Wu = (torch.randn(s, device="cuda").half() for s in ((M, K), (N, K), (N, K)))
    Wg, Wu = Wg * 0.1, Wu * 0.1
    dH = torch.randn((M, N), device="cuda")
    H, G, U = rb.qat_glu(X, Wg, Wu, h_dtype=torch.float32, save=True)
    dG, dU, _, _ = rb.qat_glu_backward(dH, G, U)
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu, dx_dtype=torch.float32)
    D = torch.randn((M, K), device="cuda").half()
    e = 2.0 ** -5
    hi, lo = (rb.qat_glu((X.float() + s * e * D.float()).half(), Wg, Wu, h_dtype=torch.float32)[0] for s in (1, -1))
    torch.cuda.synchronize()
    # the moved X is rounded to fp16 (2^-11 of values up to 5, against a step of 2^-5 times D) and the second-order rest is
    # e^2 times a third derivative of order one: a few percent of the whole
    got = float((dX.double() * D.double()).sum())
    want = float(((hi.double() - lo.double()) * dH.double()).sum() / (2 * e))
    scale = float((dX.double().abs() * D.double().abs()).sum())
    assert abs(got - want) <= 0.02 * scale


def test_update_and_decode():
    T = example()
    torch.manual_seed(2)
    b = T.GatedBlock(96, 160, planes=1, seed=5, lr=1e-2)
    emb = torch.randn((48, 96), device="cuda").to(torch.bfloat16)
    b.forward(emb)
    b.backward(torch.randn_like(emb))
    before = [y.W.double().cpu().numpy() for y in b.layers]
    grads = [y.dW.double().cpu().numpy() for y in b.layers]
    norm = float(np.sqrt(sum((g ** 2).sum() for g in grads) + sum(float(t.double().square().sum()) for t in b.dsmall)))
    b.update()
    torch.cuda.synchronize()
    for y, W, G in zip(b.layers, before, grads):
        s = 0.2 * max(W.shape) ** 0.5
        want, _, X = BO.muon(W, G, np.zeros_like(W), b.lr, 0.95, True, 0.01, s, grad_scale=min(1.0, 1.0 / norm))
        err = np.linalg.norm(y.W.double().cpu().numpy() - want)
        # X within 4e-3 (see the step's own tests), and eps against the norm scaled in fp32
        assert err <= b.lr * s * 5e-3 * np.linalg.norm(X) + 2e-7 * np.linalg.norm(W)
    b.pack(group=32)
    token = emb[:3]
    X1 = b.decode(token)
    torch.cuda.synchronize()
    w = [rb.q4_dequant(*p, *y.W.shape, group=32, dtype=torch.float32).double().cpu() for p, y in zip(b.packed, b.layers)]
    v = {k: x.double().cpu() for k, x in b.vec.items()}
    ref = reference(token.double().cpu(), *w, v)
    assert float((X1.double().cpu() - ref).norm() / ref.norm()) <= 5 * 2.0 ** -8  # X0, H, O and X1 in bf16


def test_a_bad_gradient_skips_the_step():
    b = example().GatedBlock(64, 96)
    b.forward(torch.randn((32, 64), device="cuda").to(torch.bfloat16))
    b.backward(torch.full((32, 64), float("inf"), dtype=torch.bfloat16, device="cuda"))
    kept = [t.clone() for t in [y.W for y in b.layers] + b.mom + b.small]
    b.update()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip([y.W for y in b.layers] + b.mom + b.small, kept))


def test_training_and_decoding_run():
    losses, block = example().train(tokens=64, width=128, hidden=192, steps=5)
    assert len(losses) == 5 and all(np.isfinite(losses))
    block.pack()
    assert bool(torch.isfinite(block.decode(block.emb[:1])).all())


def test_decoding_uses_the_weights_that_were_trained():
    """What is packed is the weights that the forward multiplies by, after the last update: each within half a step of
    its group's scale (W / s is rounded once before it is rounded to a code: 8 u more)."""
    T = example()
    torch.manual_seed(4)
    b = T.GatedBlock(96, 160, planes=2, seed=6, lr=1e-2)
    emb = torch.randn((48, 96), device="cuda").to(torch.bfloat16)
    b.forward(emb)
    b.backward(torch.randn_like(emb))
    b.update()
    b.pack(group=32)
    want = []
    for y in b.layers:
        y.derive()
        want.append(y.What.float().clone())
    for p, w in zip(b.packed, want):
        got = rb.q4_dequant(*p, *w.shape, group=32, dtype=torch.float32)
        s = p[1].float().t().repeat_interleave(32, 1)[:, :w.shape[1]]
        assert bool(((got - w).abs() <= s * (0.5 + 8 * 2.0 ** -24)).all())


@pytest.mark.parametrize("along", ["dX", "gate", "up"])
def test_input_gradient_against_differences(along):
    """The forward, in fp32 outputs, with X moved by D and by -D: along the whole gradient, and along each of its two terms,
    so that <dX, D> is a sum of terms of one sign. The moved X are rounded to fp16, and D is half of what then lies between
    them. What the difference and <dX, D> are apart by, of the whole: the rest of third order, e^2 / 6 = 2^-10 / 6 times a third
    derivative of the same order as the first (a part in a thousand); G, U, dG and dU rounded to fp16, 2^-11 each, over sums
    of absolute terms up to a few times the whole (under one percent); the middle of the moved X, 2^-12 of X off (less than
    that). So three percent; a dX without either term, or of the other sign, is off by about half or more."""
    torch.manual_seed(1)
    M, N, K = 64, 96, 80
    X, Wg, Wu = (torch.randn(s, device="cuda").half() for s in ((M, K), (N, K), (N, K)))
    Wg, Wu = Wg * 0.1, Wu * 0.1
    dH = torch.randn((M, N), device="cuda")
    H, G, U = rb.qat_glu(X, Wg, Wu, h_dtype=torch.float32, save=True)
    dG, dU, _, _ = rb.qat_glu_backward(dH, G, U)
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu, dx_dtype=torch.float32).double()
    gate, up = dG.double() @ Wg.double(), dU.double() @ Wu.double()
    D = {"dX": gate + up, "gate": gate, "up": up}[along]
    D = D / D.square().mean().sqrt() * 2.0 ** -5
    hi, lo = ((X.double() + s * D).half() for s in (1, -1))
    D = (hi.double() - lo.double()) / 2
    Hh, Hl = (rb.qat_glu(t, Wg, Wu, h_dtype=torch.float32)[0].double() for t in (hi, lo))
    torch.cuda.synchronize()
    want = float(((Hh - Hl) * dH.double()).sum() / 2)
    off = lambda d: abs(float((d * D).sum()) - want) / abs(want)  # noqa: E731
    assert off(dX) <= 0.03
    wrong = {"dX": (dX - gate, dX - up, -dX), "gate": (dX - gate, -dX), "up": (dX - up, -dX)}[along]
    assert all(off(d) > 0.25 for d in wrong)
