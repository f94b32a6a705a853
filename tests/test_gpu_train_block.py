"""The block of examples/train_block.py: its gradients against autograd in 64 bits, and training itself.

The gradients pass through bf16 activations and weights (unit roundoff 2^-8) several times: each tensor's
2-norm error is bounded by 2^-8 times the number of bf16 roundings on its longest path (at most 8: What,
X0, Z, H, O, dX1, dO, dH, dZ, of which no gradient sees more than 8), taken at full size.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs the GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_of_the_block():
    T = example()
    torch.manual_seed(0)
    M, D, Hd = 96, 200, 344
    b = T.Block(D, Hd, planes=2, seed=3)
    for k, v in b.vec.items():
        v.add_(torch.randn_like(v) * 0.2)
    emb = torch.randn((M, D), device="cuda").to(torch.bfloat16)
    dX1 = (torch.randn((M, D), device="cuda")).to(torch.bfloat16)
    X1 = b.forward(emb)
    demb = b.backward(dX1)
    torch.cuda.synchronize()

    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    v = {k: leaf(x) for k, x in b.vec.items()}
    up, down, e = leaf(b.up.What.float()), leaf(b.down.What.float()), leaf(emb.float())
    rms = lambda x, w: x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    z = rms(e, v["w_in"]) @ up.t() + v["bias"]
    o = (z * torch.sigmoid(z)) @ down.t()
    s1 = e + v["gate"] * rms(o, v["w_post"])
    x1 = rms(s1, v["w_out"])
    x1.backward(dX1.double().cpu())
    rel = lambda a, r: float((a.double().cpu() - r).norm() / r.norm())  # noqa: E731
    lim = 8 * 2.0 ** -8
    assert rel(X1.float(), x1.detach()) <= lim
    # the stream's gradient comes back through dR, the first norm's own through dY: their sum is in dY there
    for got, ref in ((demb.float(), e.grad), (b.up.dW, up.grad), (b.down.dW, down.grad),
                     *((b.dvec[k], v[k].grad) for k in v)):
        assert rel(got, ref) <= lim, rel(got, ref)


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss(bits):
    losses = example().train(tokens=192, width=256, hidden=512, steps=60, bits=bits)
    assert losses[-1] < 0.6 * losses[0], losses[::10]
    assert all(a == a for a in losses)


def test_a_bad_gradient_skips_the_step():
    T = example()
    b = T.Block(64, 96, bits=8)
    b.forward(torch.randn((32, 64), device="cuda").to(torch.bfloat16))
    b.backward(torch.full((32, 64), float("inf"), dtype=torch.bfloat16, device="cuda"))
    before = [p.clone() for p in b.params]
    b.update()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(b.params, before))
