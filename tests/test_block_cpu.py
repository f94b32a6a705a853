"""The training block's operators without a GPU: refusals of the C ABI (before any HIP call), the
optimizer's plan image, and pins of the oracle (worked values, differences, planted mistakes)."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

from oracle import block_oracle as BO
from residual_binarized_weight_amd import _lib

L = _lib.lib
P, P_MIS, P_ODD = (ctypes.c_void_p(x) for x in (0x100000, 0x100004, 0x100001))
P2 = ctypes.c_void_p(0x100002)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (_lib.RB_ERR_INVALID_ARG, _lib.RB_ERR_UNSUPPORTED,
                                               _lib.RB_ERR_MISALIGNED, _lib.RB_ERR_WORKSPACE)
F32, F16, BF16 = _lib.RB_F32, _lib.RB_F16, _lib.RB_BF16


# ---------------------------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------------------------
def linear(**kw):
    a = dict(X=P, dt=BF16, M=40, ldx=8192, W=P, ldw=8192, N=64, K=8192, bias=P, act=0, R=None, ldr=0, Z=None, ldz=0, Y=P,
             ydt=BF16, ldy=64, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_qat_linear(a["X"], a["dt"], a["M"], a["ldx"], a["W"], a["ldw"], a["N"], a["K"], a["bias"], a["act"], a["R"],
                           a["ldr"], a["Z"], a["ldz"], a["Y"], a["ydt"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID),
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=1 << 31), INVALID),
    (dict(N=(1 << 28) + 1, ldy=1 << 29), INVALID), (dict(ldx=8191), INVALID), (dict(ldw=8191), INVALID),
    (dict(ldy=63), INVALID), (dict(R=P, ldr=63), INVALID), (dict(Z=P, ldz=63), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(dt=3), INVALID), (dict(ydt=-1), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(ydt=F16), UNSUPPORTED),
    (dict(X=P_ODD), MISALIGNED), (dict(W=P_ODD), MISALIGNED), (dict(Y=P_ODD), MISALIGNED),
    (dict(Y=P2, ydt=F32), MISALIGNED), (dict(bias=P2), MISALIGNED), (dict(R=P_ODD, ldr=64), MISALIGNED),
    (dict(Z=P_ODD, ldz=64), MISALIGNED), (dict(ws=P_MIS), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
])
def test_linear_rejects(kw, status):
    assert L.rb_workspace_bytes(_lib.RB_OP_QAT_LINEAR, 1, 64, 8192, 40) > 0   # the ws cases rely on it
    assert linear(**kw) == status


def linear_backward(**kw):
    a = dict(dY=P, dydt=F32, M=400, N=64, lddy=64, Z=P, dt=BF16, ldz=64, act=4, dZ=P, lddz=64, db=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_qat_linear_backward(a["dY"], a["dydt"], a["M"], a["N"], a["lddy"], a["Z"], a["dt"], a["ldz"], a["act"],
                                    a["dZ"], a["lddz"], a["db"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), INVALID), (dict(dZ=None, db=None), INVALID), (dict(Z=None), INVALID), (dict(act=9), INVALID),
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(lddy=63), INVALID), (dict(ldz=63), INVALID),
    (dict(lddz=63), INVALID), (dict(dt=F32), UNSUPPORTED), (dict(dydt=F16), UNSUPPORTED), (dict(dydt=7), INVALID),
    (dict(dY=P2), MISALIGNED), (dict(Z=P_ODD), MISALIGNED), (dict(dZ=P_ODD), MISALIGNED), (dict(db=P2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=256), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
])
def test_linear_backward_rejects(kw, status):
    assert linear_backward(**kw) == status


def resnorm(**kw):
    a = dict(Y=P, dt=BF16, M=4, D=64, ldy=64, R=P, sdt=F32, ldr=64, gate=None, ldg=0, alpha=1.0, post=1, wpost=P, bpost=None,
             pre=1, wpre=P, bpre=None, eps=1e-6, S=P, lds=64, X=P, ldx=64, stats=P)
    a.update(kw)
    return L.rb_resnorm_forward(a["Y"], a["dt"], a["M"], a["D"], a["ldy"], a["R"], a["sdt"], a["ldr"], a["gate"], a["ldg"],
                                a["alpha"], a["post"], a["wpost"], a["bpost"], a["pre"], a["wpre"], a["bpre"], a["eps"],
                                a["S"], a["lds"], a["X"], a["ldx"], a["stats"], None)


SHARED = [
    (dict(M=0), INVALID), (dict(D=0), INVALID), (dict(M=1 << 31), INVALID),
    (dict(dt=4), INVALID), (dict(sdt=-1), INVALID), (dict(sdt=F16), UNSUPPORTED), (dict(post=3), INVALID),
    (dict(pre=-1), INVALID), (dict(wpost=None), INVALID), (dict(wpre=None), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(gate=P, ldg=63), INVALID), (dict(gate=P2, ldg=0), MISALIGNED), (dict(gate=P_ODD, ldg=64), MISALIGNED),
    (dict(wpost=P2), MISALIGNED), (dict(wpre=P2), MISALIGNED), (dict(bpost=P2), MISALIGNED), (dict(stats=P2), MISALIGNED),
    (dict(Y=P_ODD), MISALIGNED), (dict(S=P2), MISALIGNED), (dict(ldy=63), INVALID), (dict(lds=63), INVALID),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(Y=None), INVALID), (dict(X=None), INVALID), (dict(S=None, X=None, pre=0, wpre=None), INVALID),
    (dict(ldr=63), INVALID), (dict(ldx=63), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(R=P2), MISALIGNED), (dict(X=P_ODD), MISALIGNED), (dict(bpre=P2), MISALIGNED),
    (dict(D=16385, ldy=20000, ldr=20000, lds=20000, ldx=20000), UNSUPPORTED),
])
def test_resnorm_rejects(kw, status):
    assert resnorm(**kw) == status


def resnorm_backward(**kw):
    a = dict(dX=P, dt=BF16, M=4, D=64, lddx=64, dS=P, sdt=F32, ldds=64, Y=P, ldy=64, S=P, lds=64, stats=P, gate=None, ldg=0,
             alpha=1.0, post=1, wpost=P, bpost=None, pre=1, wpre=P, dY=P, lddy=64, dR=P, lddr=64, dgate=None, lddg=64,
             dwpost=P, dbpost=None, dwpre=P, dbpre=None, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.rb_resnorm_backward(a["dX"], a["dt"], a["M"], a["D"], a["lddx"], a["dS"], a["sdt"], a["ldds"], a["Y"], a["ldy"],
                                 a["S"], a["lds"], a["stats"], a["gate"], a["ldg"], a["alpha"], a["post"], a["wpost"],
                                 a["bpost"], a["pre"], a["wpre"], a["dY"], a["lddy"], a["dR"], a["lddr"], a["dgate"],
                                 a["lddg"], a["dwpost"], a["dbpost"], a["dwpre"], a["dbpre"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(stats=None), INVALID), (dict(dY=None), INVALID), (dict(dX=None), INVALID), (dict(S=None), INVALID),
    (dict(Y=None), INVALID), (dict(pre=0, dS=None, dwpre=None), INVALID), (dict(pre=0), INVALID),
    (dict(post=0), INVALID), (dict(dgate=P), INVALID), (dict(lddx=63), INVALID), (dict(ldds=63), INVALID),
    (dict(lddy=63), INVALID), (dict(lddr=63), INVALID), (dict(gate=P, ldg=64, dgate=P, lddg=63), INVALID),
    (dict(dX=P_ODD), MISALIGNED), (dict(dS=P2), MISALIGNED), (dict(dY=P_ODD), MISALIGNED), (dict(dR=P2), MISALIGNED),
    (dict(gate=P, dgate=P2), MISALIGNED), (dict(dwpost=P2), MISALIGNED), (dict(dwpre=P2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE), (dict(ws=P_MIS), MISALIGNED),
    (dict(D=16385, lddx=20000, ldds=20000, ldy=20000, lds=20000, lddy=20000, lddr=20000), UNSUPPORTED),
])
def test_resnorm_backward_rejects(kw, status):
    assert resnorm_backward(**kw) == status


def test_resnorm_without_a_pre_norm_takes_no_x():
    """The stream is the only output then: an X would stay unwritten, a dX would be dropped."""
    none = dict(pre=0, wpre=None)
    assert resnorm(**none) == INVALID
    assert resnorm(**none, S=None, lds=0) == INVALID
    assert resnorm(**none, X=None, S=None) == INVALID
    assert resnorm_backward(**none, dwpre=None) == INVALID
    assert resnorm_backward(**none, dwpre=None, dX=None, dS=None) == INVALID
    # what is left passes these checks and meets a later one
    assert resnorm(**none, X=None, S=P2) == MISALIGNED
    assert resnorm_backward(**none, dwpre=None, dX=None, ws=None) == WORKSPACE


def tensor(n=100, **kw):
    a = dict(p=0x100000, g=0x200000, m=0x300000, v=0x400000, m_scale=0x500000, v_scale=0x600000, n=n, lr_mult=1.0,
             weight_decay=0.1, p_dtype=F32, g_dtype=F32)
    a.update(kw)
    return _lib.AdamwTensor(*a.values())


def plan(tensors, bits=32, short=0):
    t = (_lib.AdamwTensor * max(1, len(tensors)))(*tensors)
    need = L.rb_adamw_plan_bytes(ctypes.byref(t), len(tensors))
    image, chunks = (ctypes.c_uint64 * (need // 8 + 2))(), ctypes.c_int64(-1)
    st = L.rb_adamw_plan(ctypes.byref(t), len(tensors), bits, ctypes.byref(image), need - short, ctypes.byref(chunks))
    return st, bytes(image)[:need], chunks.value


@pytest.mark.parametrize("kw,bits,status", [
    (dict(n=-1), 32, INVALID), (dict(p=None), 32, INVALID), (dict(g=None), 32, INVALID), (dict(m=None), 8, INVALID),
    (dict(v=None), 32, INVALID), (dict(m_scale=None), 8, INVALID), (dict(v_scale=None), 8, INVALID),
    (dict(lr_mult=-1.0), 32, INVALID), (dict(lr_mult=float("nan")), 32, INVALID),
    (dict(weight_decay=float("inf")), 32, INVALID), (dict(weight_decay=-0.1), 32, INVALID), (dict(p_dtype=5), 32, INVALID),
    (dict(g_dtype=-2), 32, INVALID), (dict(p_dtype=F16, g_dtype=BF16), 32, UNSUPPORTED),
    (dict(p=0x100002), 32, MISALIGNED), (dict(g=0x100001, g_dtype=F16), 32, MISALIGNED), (dict(m=0x100002), 32, MISALIGNED),
    (dict(v_scale=0x100002), 8, MISALIGNED), (dict(), 16, INVALID),
])
def test_adamw_plan_rejects(kw, bits, status):
    assert plan([tensor(), tensor(**kw)], bits)[0] == status


def test_adamw_plan_sizes_and_chunks():
    sizes = [1, 4096, 0, 4097, 12288]
    st, image, chunks = plan([tensor(n=n) for n in sizes])
    assert st == _lib.RB_OK and chunks == 1 + 1 + 0 + 2 + 3
    # header, 80 bytes a tensor, a 32-bit tensor number a chunk, whole 16 bytes
    assert len(image) == (64 + 80 * 5 + 4 * 7 + 15) // 16 * 16
    assert list(np.frombuffer(image, np.uint32)[(64 + 80 * 5) // 4:][:7]) == [0, 1, 3, 3, 4, 4, 4]
    assert plan([tensor()], short=1)[0] == WORKSPACE
    assert plan([tensor(n=0, p=None, g=None, m=None, v=None)])[::2] == (_lib.RB_OK, 0)
    assert plan([])[::2] == (_lib.RB_OK, 0)
    assert L.rb_adamw_plan_bytes(None, 1) == 0 and L.rb_adamw_plan_bytes(None, -1) == 0
    assert plan([tensor(n=1 << 62)])[0] == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), INVALID), (dict(chunks=-1), INVALID), (dict(chunks=1 << 31), INVALID), (dict(bits=4), INVALID),
    (dict(step=0), INVALID), (dict(lr=float("nan")), INVALID), (dict(lr=-1.0), INVALID), (dict(b1=1.0), INVALID),
    (dict(b1=-0.1), INVALID), (dict(b2=1.0), INVALID), (dict(b2=float("nan")), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=1e-60), INVALID), (dict(eps=float("inf")), INVALID), (dict(plan=P_MIS), MISALIGNED),
    (dict(gs=P2), MISALIGNED), (dict(skip=P2), MISALIGNED),
])
def test_adamw_step_rejects(kw, status):
    a = dict(plan=P, chunks=1, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, gs=None, skip=None)
    a.update(kw)
    assert L.rb_adamw_step(a["plan"], a["chunks"], a["bits"], a["step"], a["lr"], a["b1"], a["b2"], a["eps"], a["gs"],
                           a["skip"], 0, None) == status


def test_adamw_chunks_of_one_launch():
    """A block of 256 threads per chunk: 2^24 of them do not fit a grid, and would run short without an error."""
    most = 4096 * ((1 << 24) - 1)
    assert plan([tensor(n=most)])[::2] == (_lib.RB_OK, (1 << 24) - 1)
    assert plan([tensor(n=most + 1)])[0] == UNSUPPORTED
    assert plan([tensor(n=most), tensor(n=1)])[0] == UNSUPPORTED
    assert L.rb_adamw_step(P, 1 << 24, 32, 1, 1e-3, 0.9, 0.99, 1e-8, None, None, 0, None) == UNSUPPORTED


def test_workspace_sizes():
    zero = lambda n: (8 * n + 255) // 256 * 256  # noqa: E731
    ws = lambda op, n, k, m: L.rb_workspace_bytes(op, 1, n, k, m)  # noqa: E731
    # few rows and whole rounds of tiles need none; a split product holds fp32 [chunks][M][N]
    assert ws(_lib.RB_OP_QAT_LINEAR, 4096, 4096, 1) == 0 and ws(_lib.RB_OP_QAT_LINEAR, 4096, 11008, 2048) == 0
    got = ws(_lib.RB_OP_QAT_LINEAR, 4096, 4096, 64) - zero(4096)
    assert got > 0 and got % (64 * 4096 * 4) == 0
    # 256 blocks of partial sums for up to 5 vectors
    assert ws(_lib.RB_OP_RESNORM_BACKWARD, 4096, 1, 2048) == zero(4096) + 5 * 256 * 4096 * 4
    assert ws(_lib.RB_OP_RESNORM_BACKWARD, 4096, 1, 3) == zero(4096) + 5 * 3 * 4096 * 4
    assert ws(_lib.RB_OP_RESNORM_BACKWARD, 16385, 1, 3) == 0
    for M, strips in ((1, 1), (5, 2), (256, 64), (257, 52), (2048, 64)):    # past 8192 columns: strips, and the rows' means
        assert ws(_lib.RB_OP_RESNORM_BACKWARD, 9000, 1, M) == zero(9000) + 5 * strips * 9000 * 4 + 16 * M
    assert ws(_lib.RB_OP_QAT_LINEAR_BACKWARD, 512, 1, 8) == 0       # one strip: its sums are db
    got = ws(_lib.RB_OP_QAT_LINEAR_BACKWARD, 512, 1, 9) - zero(512)
    assert got > 0 and got % (512 * 4) == 0


def test_product_workspace_follows_the_layout_rule():
    """The partial sums of the layout that the restated rule chooses, over 6000 shapes; 256-row tiles first where small
    tiles alone are not clearly estimated below them (312 x 33832 x 1024 and 617 x 25264 x 4096 are whole, where 256-row
    tiles would leave a rest with split columns)."""
    from tests import linear_forms as F
    r = np.random.default_rng(40)
    draw = lambda lo, hi: np.exp(r.uniform(np.log(lo), np.log(hi), 6000)).round().astype(int)  # noqa: E731
    shapes = list(zip(draw(1, 8192), draw(1, 40000), draw(1, 12000)))
    shapes += [(M, (N + 7) // 8 * 8, (K + 7) // 8 * 8) for M, N, K in shapes[:2000]]
    shapes += [(312, 33832, 1024), (617, 25264, 4096), (1654, 9712, 3608), (2048, 11008, 4096), (2048, 4096, 11008)]
    for M, N, K in shapes:
        w = F.workspace(int(M), int(N), int(K))
        assert L.rb_workspace_bytes(_lib.RB_OP_QAT_LINEAR, 1, int(N), int(K), int(M)) == (w and w + (8 * int(N) + 255) // 256 * 256)
    assert F.tiles(312, 33832, 1024, True)[1] == 0 and F.tiles(617, 25264, 4096, True)[1] == 0
    assert F.form(2550, 9640, 2064, True) == "128" and F.form(2048, 11008, 4096, True) == "256+128"


# ---------------------------------------------------------------------------------------------
# the oracle's own pins
# ---------------------------------------------------------------------------------------------
def test_oracle_worked_values():
    Y, Z = BO.linear([[1.0, 2.0]], [[3.0, -1.0], [0.5, 0.25]], bias=[0.0, -2.0], act="relu", residual=[[10.0, 20.0]])
    assert Z.tolist() == [[1.0, -1.0]] and Y.tolist() == [[11.0, 20.0]]
    assert BO.linear_backward([[2.0, 3.0, 1.0]], [[1.0, -1.0, 0.0]], "relu")[0].tolist() == [[2.0, 0.0, 0.0]]
    # rows (3, 4): mean square 12.5; centred (-1/2, 1/2): variance 1/4
    S, X, st = BO.resnorm([[3.0, 4.0]], [[1.0, 1.0]], [2.0, 2.0], gate=[1.0, 0.5], alpha=2.0, eps=0.0, pre="layer")
    assert S.tolist() == [[5.0, 4.0]] and X.tolist() == [[2.0, -2.0]] and st.tolist() == [[0.0, 0.0, 4.5, 2.0]]
    assert np.allclose(BO.norm([[3.0, 4.0]], "rms", [1.0, 1.0], [0.5, 0.0], 0.0), np.array([[3, 4]]) / 12.5 ** 0.5 + [[0.5, 0]])
    # first step from zero: m / (1 - b1) = g, sqrt(v / (1 - b2)) = |g|: a step of lr against the sign
    p, m, v = BO.adamw([1.0, 1.0], [0.5, -2.0], [0.0, 0.0], [0.0, 0.0], 1, 0.1, 0.9, 0.99, 0.0, 0.0)
    assert np.allclose(p, [0.9, 1.1]) and np.allclose(m, [0.05, -0.2]) and np.allclose(v, [0.0025, 0.04])
    assert np.isclose(BO.adamw([1.0], [0.0], [0.0], [0.0], 1, 0.1, weight_decay=0.5)[0][0], 0.95)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_oracle_slopes_are_differences(act):
    z = np.linspace(-6, 6, 241) + 0.0123
    h = 1e-5
    diff = (BO.activation(z + h, act)[0] - BO.activation(z - h, act)[0]) / (2 * h)
    assert np.max(np.abs(diff - BO.activation(z, act)[1])) < 1e-8


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", 1), ("layer", "layer", 2), ("none", "rms", 0), ("rms", "none", 1)])
def test_oracle_norm_gradients_are_differences(post, pre, gate):
    r = np.random.default_rng(5)
    M, D, eps, h = 3, 7, 1e-3, 1e-6
    a = dict(Y=r.standard_normal((M, D)), R=r.standard_normal((M, D)), w_pre=r.random(D) + 0.5, w_post=r.random(D) + 0.5,
             b_pre=r.standard_normal(D), b_post=r.standard_normal(D) if post != "none" else None,
             gate=[None, r.standard_normal(D), r.standard_normal((M, D))][gate])
    kw = dict(alpha=0.7, pre=pre, post=post)
    S, X, st = BO.resnorm(**a, eps=eps, **kw)
    dX = r.standard_normal((M, D)) if pre != "none" else None
    dS = r.standard_normal((M, D))
    g = BO.resnorm_backward(dX, dS, a["Y"], S, st, a["w_pre"], a["w_post"], a["b_post"], a["gate"], **kw)

    def loss(b):
        s, x, _ = BO.resnorm(**b, eps=eps, **kw)
        return (s * dS).sum() + (0 if x is None else (x * dX).sum())
    for k, gk in dict(Y="dY", R="dR", w_pre="dw_pre", w_post="dw_post", b_pre="db_pre", b_post="db_post", gate="dgate").items():
        if g[gk] is None or a[k] is None:
            continue
        v = r.standard_normal(a[k].shape)
        diff = (loss({**a, k: a[k] + h * v}) - loss({**a, k: a[k] - h * v})) / (2 * h)
        assert abs(diff - (g[gk] * v).sum()) < 1e-6 * (1 + abs(diff)), k


def test_oracle_8bit_codes():
    assert BO.E4M3[0x38] == 1.0 and BO.E4M3[0x78] == 256.0 and BO.E4M3[0x01] == 2.0 ** -9 and BO.E4M3[0xB8] == -1.0
    assert np.isnan(BO.E4M3[0x7F]) and BO.E4M3[0x7E] == 448.0
    assert BO.adamw_scales(np.array([0.75, -1.0, 0.0])).tolist() == [2.0]
    assert BO.adamw_scales(np.zeros(300)).tolist() == [2.0 ** -99] * 2
    # every positive code of a group is on the grid of its scale
    x = BO.adamw_decode(np.arange(0x78, dtype=np.uint8), [1.0])
    a, grid = BO.adamw_grid(x, np.array([1.0]))
    assert np.array_equal(a, BO.E4M3[:0x78]) and np.all(a / grid == np.floor(a / grid))
    h = BO.adamw_random(np.arange(4096), 3, 11)
    for half in (h & 0xFFFF, h >> 16):   # uniform: mean and spread within 5 deviations
        assert abs(half.mean() - 32767.5) < 5 * 18918 / 64 and abs(half.std() - 18918) < 5 * 18918 / 64 / 1.5


MUTANTS = {
    "relu_slope_at_zero": ("(z > 0).astype", "(z >= 0).astype"),
    "bias_after_activation": ("    Y = activation(Z, act)[0]\n", "    Y = activation(Z - (0 if bias is None else _f(bias)), act)[0]\n"),
    "norm_gradient_without_projection": ("dx = d - xh * (d * xh).mean(axis=1, keepdims=True)", "dx = d"),
    "layer_gradient_without_mean": ("        dx = dx - d.mean(axis=1, keepdims=True)\n", "        pass\n"),
    "eps_outside_the_root": (".mean(axis=1) + eps)", ".mean(axis=1)) + eps"),
    "alpha_not_in_dr": ('out["dR"] = alpha * T', 'out["dR"] = T'),
    "gate_after_post_gradient": ("        du = _f(gate) * T\n", "        du = T\n"),
    "decay_into_the_moments": ("g = _f(p), _f(g) * grad_scale", "g = _f(p), _f(g) * grad_scale + weight_decay * _f(p)"),
    "no_bias_correction": ("(m / (1.0 - beta1 ** step))", "m"),
    "scale_not_above_the_largest": ("[1])\n\n\ndef adamw_grid", "[1] - 1)\n\n\ndef adamw_grid"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_oracle_pins_catch(name, tmp_path):
    """A mistake planted in a copy of the oracle fails one of the pins above."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    old, new = MUTANTS[name]
    for d in ("oracle", "tests"):
        os.makedirs(tmp_path / d)
    for f in ("oracle/__init__.py", "oracle/rb_oracle.py", "oracle/block_oracle.py", "tests/test_block_cpu.py", "tests/conftest.py"):
        shutil.copy(os.path.join(root, f), tmp_path / f)
    os.symlink(os.path.join(root, "residual_binarized_weight_amd"), tmp_path / "residual_binarized_weight_amd")
    src = (tmp_path / "oracle/block_oracle.py").read_text()
    assert src.count(old) == 1, f"{name}: the planted line is not there once"
    (tmp_path / "oracle/block_oracle.py").write_text(src.replace(old, new))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_block_cpu.py",
                        "-k", "oracle and not pins_catch"], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 1, f"{name} was not caught:\n{r.stdout[-600:]}"
