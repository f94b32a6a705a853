"""The gated block's operators, without a GPU: their oracle against autograd, differences and worked examples, the
refusals of their C entry points, and their workspaces."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import residual_binarized_weight_amd as rb
from oracle import block_oracle as BO
from residual_binarized_weight_amd import _lib

L = _lib.lib
P, P2, P_ODD, P_MIS = (ctypes.c_void_p(0x100000 + i) for i in (0, 2, 1, 4))
F32, F16, BF16 = _lib.RB_F32, _lib.RB_F16, _lib.RB_BF16
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (_lib.RB_ERR_INVALID_ARG, _lib.RB_ERR_UNSUPPORTED, _lib.RB_ERR_MISALIGNED,
                                               _lib.RB_ERR_WORKSPACE)
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# --------------------------------------------------------------------------------------------
# oracle
# --------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
def test_glu_gradients_against_autograd_and_differences(act):
    r = np.random.default_rng(5)
    M, N, K = 5, 7, 6
    X, Wg, Wu = r.standard_normal((M, K)), r.standard_normal((N, K)), r.standard_normal((N, K))
    bg, bu, dH = r.standard_normal(N), r.standard_normal(N), r.standard_normal((M, N))
    leaf = [torch.from_numpy(t).requires_grad_() for t in (X, Wg, Wu, bg, bu)]
    f = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act]
    h = f(leaf[0] @ leaf[1].t() + leaf[3]) * (leaf[0] @ leaf[2].t() + leaf[4])
    h.backward(torch.from_numpy(dH))
    H, G, U = BO.glu(X, Wg, Wu, bg, bu, act)
    np.testing.assert_allclose(H, h.detach().numpy(), rtol=1e-12, atol=1e-12)
    dG, dU, dbg, dbu = BO.glu_backward(dH, G, U, act)
    got = (BO.glu_dx(dG, dU, Wg, Wu), dG.T @ X, dU.T @ X, dbg, dbu)
    for a, b in zip(got, leaf):
        np.testing.assert_allclose(a, b.grad.numpy(), rtol=1e-11, atol=1e-12)
    # the whole directional derivative, by central differences
    step = [r.standard_normal(t.shape) for t in (X, Wg, Wu, bg, bu)]
    at = lambda e: (BO.glu(*(t + e * d for t, d in zip((X, Wg, Wu, bg, bu), step)), act)[0] * dH).sum()  # noqa: E731
    e = 1e-6
    assert (at(e) - at(-e)) / (2 * e) == pytest.approx(sum((g * d).sum() for g, d in zip(got, step)), rel=1e-6, abs=1e-6)


@pytest.mark.parametrize("N,K", [(6, 9), (9, 6), (8, 8), (1, 5), (5, 1)])
def test_newton_schulz_against_its_products(N, K):
    r = np.random.default_rng(7)
    u = r.standard_normal((N, K))
    X = u / (np.linalg.norm(u) + 1e-7)
    a, b, c = BO.NS_COEFFICIENTS
    for _ in range(5):
        A = X @ X.T
        X = a * X + (b * A + c * A @ A) @ X
    np.testing.assert_allclose(BO.newton_schulz(u), X, rtol=1e-9, atol=1e-11)
    s = np.linalg.svd(BO.newton_schulz(u), compute_uv=False)
    assert np.all((s > 0.3) & (s < 1.3))


def test_newton_schulz_of_nothing_is_nothing():
    assert not BO.newton_schulz(np.zeros((3, 4))).any()


def test_polynomial_stays_within_the_held_range():
    """The fixed powers of two that the products' operands are held at rest on these bounds: singular values start at
    most 1 and never pass 1.21; A's stay below 1.47 and those of b A + c A^2 within 2.81."""
    a, b, c = BO.NS_COEFFICIENTS
    s = np.linspace(0, 1.21, 200001)
    assert (a * s + b * s ** 3 + c * s ** 5).max() <= 1.21 and (a * s + b * s ** 3 + c * s ** 5).min() >= 0
    assert 1.21 ** 2 < 1.47
    t = np.linspace(0, 1.47, 200001)
    assert np.abs(b * t + c * t * t).max() < 2.81
    assert 1.21 * 2 ** 15 < 65504 and 1.47 * 2 ** 15 < 65504 and 2.81 * 2 ** 14 < 65504


def test_muon_by_hand():
    # one row: X is the row over its norm taken through the scalar polynomial
    W, G, m = np.array([[1.0, 2.0]]), np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]])
    a, b, c = BO.NS_COEFFICIENTS
    x = 1.0
    for _ in range(5):
        x = a * x + b * x ** 3 + c * x ** 5
    W2, m2, X = BO.muon(W, G, m, 0.1, 0.5, True, 0.2, 2.0, eps=1e-30)
    np.testing.assert_allclose(m2, [[3.0, 4.0]])
    np.testing.assert_allclose(X, [[0.6 * x, 0.8 * x]], rtol=1e-12)
    np.testing.assert_allclose(W2, W * 0.98 - 0.2 * X, rtol=1e-12)


def test_q4_by_hand():
    w = np.array([[7.0, -7.0, 3.4, 3.5, 4.5, 0.0, -0.5, 0.5]], dtype=np.float32)
    q, s, z = BO.q4_quantise(w, 32, False)
    assert s[0, 0] == 1.0 and z is None
    assert q.tolist() == [[15, 1, 11, 12, 12, 8, 8, 8]]  # ties to even
    q, s, z = BO.q4_quantise(w + 7, 32, True)
    assert z[0, 0] == 0.0 and s[0, 0] == np.float16(14 / 15)
    np.testing.assert_allclose(BO.q4_values(q, s, z, 32), w + 7, atol=0.5 * 14 / 15 + 1e-2)


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (17, 130, 32), (33, 300, 64), (16, 256, 128)])
def test_q4_layout_round_trip(N, K, group):
    q = np.random.default_rng(3).integers(0, 16, (N, K))
    w = BO.q4_codes(q)
    assert w.nbytes == L.rb_q4_codes_bytes(N, K)
    for n, c in ((0, 0), (N - 1, K - 1), (N // 2, K // 3)):
        word = int(w[n // 16, c // 128, 16 * (c // 8 % 4) + n % 16, c // 32 % 4])
        assert word >> (16 * (c % 2) + 4 * (c % 8 // 2)) & 15 == q[n, c]
    assert int(w.astype(np.uint64).sum()) == sum(int(v) << (16 * (c % 2) + 4 * (c % 8 // 2)) for (n, c), v in np.ndenumerate(q))


# --------------------------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------------------------
def _glu(**kw):
    a = dict(X=P, dt=BF16, M=300, ldx=6400, Wg=P, ldwg=6400, Wu=P, ldwu=6400, N=520, K=6400, bg=None, bu=None, act=4, G=None, ldg=520,
             U=None, ldu=520, H=P, hdt=BF16, ldh=520, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_qat_glu(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    *((dict([(k, None)]), INVALID) for k in ("X", "Wg", "Wu", "H")),
    *((dict([(k, 0)]), INVALID) for k in ("M", "N", "K")),
    (dict(N=(1 << 28) + 1, ldh=1 << 29), INVALID), (dict(K=(1 << 28) + 1, ldx=1 << 29, ldwg=1 << 29, ldwu=1 << 29), INVALID),
    (dict(M=1 << 31), INVALID),
    *((dict([(k, 6399)]), INVALID) for k in ("ldx", "ldwg", "ldwu")),
    *((dict([(k, 1 << 31)]), INVALID) for k in ("ldx", "ldwg", "ldwu", "ldh")),
    (dict(ldh=519), INVALID), (dict(G=P, ldg=519), INVALID), (dict(U=P, ldu=519), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(dt=9), INVALID), (dict(hdt=-1), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(hdt=F16), UNSUPPORTED),
    (dict(M=(1 << 31) - 1, N=1 << 28, ldh=1 << 28), UNSUPPORTED),
    *((dict([(k, P_ODD)]), MISALIGNED) for k in ("X", "Wg", "Wu", "H", "G", "U")),
    (dict(H=P2, hdt=F32), MISALIGNED), (dict(bg=P2), MISALIGNED), (dict(bu=P2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
])
def test_glu_rejects(kw, status):
    assert _glu(**kw) == status


def _glu_backward(**kw):
    a = dict(dH=P, hdt=BF16, M=300, N=64, lddh=64, G=P, ldg=64, U=P, ldu=64, dt=BF16, act=4, dG=P, lddg=64, dU=P2, lddu=64,
             dbg=P, dbu=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_qat_glu_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    *((dict([(k, None)]), INVALID) for k in ("dH", "G", "U", "dG", "dU")),
    (dict(dU=P), INVALID),  # both gradients in one place
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(M=1 << 31), INVALID),
    *((dict([(k, 63)]), INVALID) for k in ("lddh", "ldg", "ldu", "lddg", "lddu")),
    (dict(act=7), INVALID), (dict(dt=5), INVALID), (dict(hdt=5), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(hdt=F16), UNSUPPORTED),
    *((dict([(k, P_ODD)]), MISALIGNED) for k in ("dH", "G", "U", "dG", "dU")),
    (dict(dH=P2, hdt=F32), MISALIGNED), (dict(dbg=P2), MISALIGNED), (dict(dbu=P2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws=None, dbu=None), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
])
def test_glu_backward_rejects(kw, status):
    assert _glu_backward(**kw) == status


def _glu_dx(**kw):
    a = dict(dG=P, lddg=5200, dU=P, lddu=5200, dt=BF16, M=300, Wg=P, ldwg=64, Wu=P, ldwu=64, N=5200, K=64, dX=P, xdt=BF16,
             lddx=64, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_qat_glu_dx(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    *((dict([(k, None)]), INVALID) for k in ("dG", "dU", "Wg", "Wu", "dX")),
    *((dict([(k, 0)]), INVALID) for k in ("M", "N", "K")),
    *((dict([(k, 63)]), INVALID) for k in ("ldwg", "ldwu", "lddx")), (dict(lddg=5199), INVALID), (dict(lddu=5199), INVALID),
    (dict(dt=4), INVALID), (dict(xdt=4), INVALID), (dict(dt=F32), UNSUPPORTED), (dict(xdt=F16), UNSUPPORTED),
    *((dict([(k, P_ODD)]), MISALIGNED) for k in ("dG", "dU", "Wg", "Wu", "dX")), (dict(dX=P2, xdt=F32), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=300), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
])
def test_glu_dx_rejects(kw, status):
    assert _glu_dx(**kw) == status


def _muon(**kw):
    a = dict(W=P, ldw=64, G=P, gdt=F32, ldg=64, mom=P, ldm=64, N=40, K=64, lr=1e-3, mu=0.9, nesterov=1, wd=0.1, scale=1.0,
             steps=5, eps=1e-7, gs=None, skip=None, O=None, odt=F16, ldo=64, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_muon_step(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), INVALID), (dict(W=None), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(N=1 << 21), INVALID), (dict(K=1 << 21, ldw=1 << 21, ldg=1 << 21, ldm=1 << 21), INVALID),
    *((dict([(k, 63)]), INVALID) for k in ("ldw", "ldg", "ldm")), (dict(O=P, ldo=63), INVALID),
    *((dict([(k, v)]), INVALID) for k in ("lr", "wd", "scale") for v in (-1.0, math.inf, math.nan)),
    (dict(mu=1.0), INVALID), (dict(mu=-0.1), INVALID), (dict(mu=math.nan), INVALID),
    (dict(steps=0), INVALID), (dict(steps=17), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=1e-60), INVALID), (dict(eps=math.inf), INVALID),
    (dict(gdt=3), INVALID), (dict(O=P, odt=3), INVALID), (dict(O=P, odt=F32), UNSUPPORTED),
    *((dict([(k, P2)]), MISALIGNED) for k in ("W", "G", "mom", "gs", "skip")), (dict(G=P_ODD, gdt=BF16), MISALIGNED),
    (dict(O=P_ODD), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=1000), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
])
def test_muon_rejects(kw, status):
    assert _muon(**kw) == status


def _q4(fn, **kw):
    a = dict(codes=P, s=P, z=None, N=40, K=200, group=64, x=P, dt=BF16, M=3, ldx=200, y=P, ydt=BF16, ldy=40)
    if fn == "glu":
        a = dict(codes=P, s=P, z=None, codes2=P, s2=P, z2=None, N=40, K=200, group=64, act=4, x=P, dt=BF16, M=3, ldx=200, y=P,
                 ydt=BF16, ldy=40)
    if fn == "pack":
        a = dict(x=P, dt=F32, N=40, K=200, ldx=200, group=64, codes=P, s=P, z=None, status=None)
    if fn == "dequant":
        a = dict(codes=P, s=P, z=None, N=40, K=200, group=64, x=P, dt=BF16, ldx=200)
    a.update(kw)
    return {"gemv": L.rb_q4_gemv, "glu": L.rb_q4_glu, "pack": L.rb_q4_pack, "dequant": L.rb_q4_dequant}[fn](*a.values(), None)


@pytest.mark.parametrize("fn", ["gemv", "glu", "pack", "dequant"])
@pytest.mark.parametrize("kw,status", [
    *((dict([(k, None)]), INVALID) for k in ("codes", "s", "x")), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(N=(1 << 28) + 1, ldy=1 << 29), INVALID), (dict(K=(1 << 28) + 1, ldx=1 << 29), INVALID),
    (dict(group=16), INVALID), (dict(group=0), INVALID), (dict(group=256), INVALID), (dict(group=96), INVALID),
    (dict(ldx=199), INVALID), (dict(dt=7), INVALID),
    (dict(codes=ctypes.c_void_p(0x100008)), MISALIGNED), (dict(s=P_ODD), MISALIGNED), (dict(z=P_ODD), MISALIGNED), (dict(x=P_ODD), MISALIGNED),
])
def test_q4_rejects(fn, kw, status):
    kw = {k: v for k, v in kw.items() if k != "ldy" or fn in ("gemv", "glu")}
    assert _q4(fn, **kw) == status


@pytest.mark.parametrize("fn", ["gemv", "glu"])
@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INVALID), (dict(M=0), INVALID), (dict(ldy=39), INVALID), (dict(ydt=5), INVALID),
    (dict(M=17), UNSUPPORTED), (dict(dt=F32), UNSUPPORTED), (dict(ydt=F16), UNSUPPORTED),
    (dict(y=P_ODD), MISALIGNED), (dict(y=P2, ydt=F32), MISALIGNED),
])
def test_q4_product_rejects(fn, kw, status):
    assert _q4(fn, **kw) == status


def test_q4_glu_and_pack_reject_their_own():
    assert _q4("glu", act=5) == INVALID and _q4("glu", codes2=None) == INVALID and _q4("glu", s2=None) == INVALID
    assert _q4("glu", z2=P_ODD) == MISALIGNED
    assert _q4("pack", status=P2) == MISALIGNED and _q4("pack", x=P2) == MISALIGNED


def test_workspaces():
    W = lambda op, N, K, M, k=1: int(L.rb_workspace_bytes(op, k, N, K, M))  # noqa: E731
    assert W(_lib.RB_OP_QAT_GLU, 11008, 4096, 1) == 0 and W(_lib.RB_OP_QAT_GLU, 1 << 29, 8, 8) == 0
    assert W(_lib.RB_OP_QAT_GLU, 520, 6400, 300) > 0 and W(_lib.RB_OP_QAT_GLU_DX, 5200, 64, 300) > 0
    assert W(_lib.RB_OP_QAT_GLU_BACKWARD, 1000, 1, 8) == 0 and W(_lib.RB_OP_QAT_GLU_BACKWARD, 1000, 1, 9) > 0
    # X in two halves twice, A and B, and the partial sums
    assert W(_lib.RB_OP_MUON_STEP, 128, 256, 1) >= 8 * 128 * 256 + 4 * 128 * 128
    assert W(_lib.RB_OP_MUON_STEP, 1 << 21, 8, 1) == 0
    assert L.rb_q4_codes_bytes(17, 129) == 2 * 2 * 1024 and L.rb_q4_codes_bytes(0, 1) == 0


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rb.qat_glu(x, x, x[:3])
    with pytest.raises(ValueError):
        rb.qat_glu_dx(x, x, x, x)
    with pytest.raises(ValueError):
        rb.q4_pack(x, group=48)
    with pytest.raises(TypeError):
        rb.muon_step(x, x, None, 0.1, grad_scale=x)
    with pytest.raises(ValueError):
        rb.q4_gemv(torch.zeros(3, dtype=torch.int32), x, None, x, 4)


def test_backward_without_dx_still_refuses():
    a = dict(dY=P, dt=BF16, M=4, lddy=16, X=P, ldx=64, What=P, ldwh=64, planes=P, ldp=2, g=P, h=P, k=2, N=16, K=64, dW=P, lddw=64,
             dX=None, xdt=BF16, lddx=0, dg=P, dh=P, ws=None, wsb=0)
    assert L.rb_qat_backward(*a.values(), None) == INVALID        # this one needs a dX
    a.update(dX=P)
    assert L.rb_qat_backward(*a.values(), None) == INVALID        # and its leading dimension
    w = {n: v for n, v in a.items() if n not in ("dX", "xdt", "lddx")}
    assert L.rb_qat_backward_weights(*w.values(), None) == WORKSPACE
    for bad in (dict(dY=None), dict(X=None), dict(dW=None), dict(dg=None), dict(dh=None), dict(M=0), dict(lddw=63)):
        assert L.rb_qat_backward_weights(*{**w, **bad}.values(), None) == INVALID


def test_inline_assembly_leaves_m0_to_the_compiler():
    """m0 is no register that a statement can list as clobbered: one that needs it takes it as an input."""
    src = os.path.join(os.path.dirname(rb.__file__), "csrc")
    for name in sorted(os.listdir(src)):
        with open(os.path.join(src, name)) as f:
            text = f.read()
        assert not re.search(r"\bs_\w+\s+m0\s*,", text), name


@pytest.mark.parametrize("kw", [dict(lr=1e30, scale=1e30), dict(lr=1e30, wd=1e30), dict(lr=1e200, scale=1e200),
                                dict(lr=1e200, wd=1e200), dict(eps=1e39)])
def test_muon_rejects_factors_past_fp32(kw):
    """With no gradient X is 0 and W has to stay: an infinite rate times X would be NaN."""
    assert _muon(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(lr=1e30, scale=1e8), dict(lr=1e30, wd=1e8), dict(eps=3e38)])
def test_muon_takes_factors_within_fp32(kw):
    assert _muon(**kw, ws=None) == WORKSPACE  # the next check


@pytest.mark.parametrize("group", [0, -32, 48, 256])
def test_q4_wrappers_refuse_other_groups(group):
    w = (torch.zeros((1, 1, 64, 4), dtype=torch.int32), torch.zeros((1, 16), dtype=torch.float16), None)
    x = torch.zeros((1, 128), dtype=torch.float16)
    for call in (lambda: rb.q4_gemv(*w, x, 16, group=group), lambda: rb.q4_glu(w, w, x, 16, group=group),
                 lambda: rb.q4_dequant(*w, 16, 128, group=group), lambda: rb.q4_pack(x, group=group)):
        with pytest.raises(ValueError, match="group"):
            call()
