"""GPU parity of the gated block's first half (rb_qat_glu), of its epilogue's backward (rb_qat_glu_backward) and of the
input's gradient (rb_qat_glu_dx) against the oracle.

Comparison rules, u = 2^-24:
* G, U: the products of fp16/bf16 numbers are exact in fp32; they are added 32 to a matrix instruction and K / 32
  instructions deep, a split tile's parts (at most 256) after that in order, the bias last: within (K / 32 + 300) u of
  S = sum |x w| + |b| where tiles may be split, whose parts are few unless K is long; the vector units' form adds K / 64
  terms a lane, then 64 lanes: below that;
* H: act has a slope below 1.13 and its evaluation is within 16 u of |g| + |act(g)|; the product and the factors' errors;
* dG, dU: slope within 24 u (1 + |g|), value within 16 u (|g| + |act(g)|), three products' roundings; their sums those
  errors and M u of the sum of |terms|;
* dX: as G, with 2 N terms;
* rounded outputs add half a unit of their type.
"""
import numpy as np
import pytest
import torch

import residual_binarized_weight_amd as rb
from oracle import block_oracle as BO
from tests.gpu_util import dev, long_buffer, pieces

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs the GPU")]

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def n64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def mat(r, M, N, dt, std=1.0, pad=0, off=0):
    """M rows of N, pad elements between them and off before; what lies between is NaN: a kernel that
    reads it shows."""
    buf = torch.full((M * (N + pad) + off,), float("nan"), dtype=DT[dt], device=dev())
    v = buf[off:].view(M, N + pad)[:, :N]
    v.copy_(torch.from_numpy((r.standard_normal((M, N)) * std).astype(np.float32)).to(DT[dt]).to(dev()))
    return v


def out(M, N, dt, pad=0, off=0):
    """A strided output and the buffer that it lies in, filled with a mark."""
    buf = torch.full((M * (N + pad) + off,), 77.0, dtype=DT[dt], device=dev())
    return buf[off:].view(M, N + pad)[:, :N], buf


def untouched(v, buf, M, N, pad, off):
    v.fill_(77.0)
    assert bool((buf == 77.0).all()), "written outside the rows"


def near(got, ref, lim, what):
    lim = lim + UNIT[got.dtype] * np.abs(ref) + TINY[got.dtype]
    err = np.abs(n64(got) - ref)
    assert np.all(err <= lim), f"{what}: {np.nanmax(err / lim):.3g} x the bound, {np.isnan(err).sum()} NaN"


def check(X, Wg, Wu, bg, bu, act, H, G, Uu):
    x, wg, wu = n64(X), n64(Wg), n64(Wu)
    h, g, u = BO.glu(x, wg, wu, n64(bg), n64(bu), act)
    K = x.shape[1]
    lg, lu = ((K / 32 + 300) * U * (np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(n64(b)))) for w, b in ((wg, bg), (wu, bu)))
    if G is not None:
        near(G, g, lg, "G")
    if Uu is not None:
        near(Uu, u, lu, "U")
    a = BO.activation(g, act)[0]
    la = 1.13 * lg + 16 * U * (np.abs(g) + np.abs(a))
    near(H, h, la * (np.abs(u) + lu) + np.abs(a) * lu + 2 * U * np.abs(h), "H")


def case(seed, M, N, K, dt, act="silu", bias=False, hdt=None, save=False, pad=0, off=0):
    r = np.random.default_rng([930, seed])
    hdt = hdt or dt
    X, Wg, Wu = mat(r, M, K, dt, 1.0, pad, off), mat(r, N, K, dt, 0.05, pad, off), mat(r, N, K, dt, 0.05, pad, off)
    bg, bu = (torch.from_numpy(r.standard_normal(N).astype(np.float32)).to(dev()) if bias else None for _ in range(2))
    outs = [out(M, N, t, pad, off) for t in (hdt, dt, dt)]
    H, G, Uu = rb.qat_glu(X, Wg, Wu, act=act, bias_g=bg, bias_u=bu, H=outs[0][0], G=outs[1][0] if save else None,
                          U=outs[2][0] if save else None)
    torch.cuda.synchronize()
    check(X, Wg, Wu, bg, bu, act, H, G, Uu)
    assert (G is not None) == save
    for v, buf in outs:
        untouched(v, buf, M, N, pad, off)


# sizes around every tile edge: 64, 128 and 256 batch rows, 32, 64 and 128 outputs, steps of 64 columns
@pytest.mark.parametrize("M", [1, 2, 4, 5, 63, 64, 65, 128, 130, 257])
@pytest.mark.parametrize("N,K", [(1, 8), (31, 64), (32, 72), (128, 128), (129, 136), (300, 1000)])
def test_tile_edges(M, N, K):
    case(1, M, N, K, "bf16", bias=True, hdt="f32", save=True)


@pytest.mark.parametrize("M", [1, 3, 5, 64, 100, 130])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (64, 7), (63, 9), (64, 63), (257, 65), (100, 997)])
def test_tile_edges_unaligned(M, N, K):
    case(2, M, N, K, "f16", bias=True, hdt="f32", save=True)


# the same where more rows, or longer ones, bring the tiles
@pytest.mark.parametrize("M", [257, 271, 320, 385])
@pytest.mark.parametrize("N,K", [(1, 8), (31, 64), (129, 72), (300, 1000)])
def test_tile_edges_of_more_rows(M, N, K):
    case(7, M, N, K, "bf16", bias=True, hdt="f32", save=True)


@pytest.mark.parametrize("M", [257, 300, 400])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (64, 7), (63, 9), (130, 63), (100, 997)])
def test_tile_edges_unaligned_of_more_rows(M, N, K):
    case(8, M, N, K, "f16", bias=True, hdt="f32", save=True)


@pytest.mark.parametrize("M", [5, 20, 64, 100])
@pytest.mark.parametrize("N,K", [(33, 20000), (129, 20001), (2000, 4104)])
def test_long_rows(M, N, K):
    case(9, M, N, K, "bf16", bias=True, hdt="f32", save=True)


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (0, 1), (1, 5)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 200), (3, 1032), (40, 264), (150, 328), (300, 264), (40, 9000)])
def test_strides_and_offsets(pad, off, dt, M, K):
    case(3, M, 70, K, dt, bias=True, save=True, pad=pad, off=off)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,hdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("bias,save", [(False, False), (True, True)])
def test_epilogues(act, dt, hdt, bias, save):
    case(4, 2, 130, 160, dt, act, bias, hdt, save)
    case(5, 37, 130, 160, dt, act, bias, hdt, save)
    case(6, 270, 130, 160, dt, act, bias, hdt, save)   # tiles
    case(10, 37, 260, 20000, dt, act, bias, hdt, save)  # split tiles: the join's epilogue


# rows enough for the 256-row tiles, a rest that is split, and rounds of whole tiles with a rest
@pytest.mark.parametrize("M,N,K", [(512, 1024, 512), (700, 1100, 2048), (2100, 4200, 128), (1024, 8192, 200), (515, 33000, 64)])
@pytest.mark.parametrize("aligned", [True, False])
def test_many_tiles(M, N, K, aligned):
    r = np.random.default_rng([931, M])
    X, Wg, Wu = (mat(r, n, K, "bf16", s, 0 if aligned else 1) for n, s in ((M, 1.0), (N, 0.05), (N, 0.05)))
    H, G, Uu = rb.qat_glu(X, Wg, Wu, save=True)
    torch.cuda.synchronize()
    rows = np.unique(np.r_[0, M - 1, r.integers(0, M, 40)])
    at = torch.from_numpy(rows).to(dev())
    check(X[at], Wg, Wu, None, None, "silu", H[at], G[at], Uu[at])


def test_one_weight_without_the_other_bias():
    r = np.random.default_rng(932)
    for M in (2, 20):
        X, Wg, Wu = mat(r, M, 96, "bf16"), mat(r, 40, 96, "bf16", 0.1), mat(r, 40, 96, "bf16", 0.1)
        b = torch.from_numpy(r.standard_normal(40).astype(np.float32)).to(dev())
        for bg, bu in ((b, None), (None, b)):
            H, G, _ = rb.qat_glu(X, Wg, Wu, act="gelu", bias_g=bg, bias_u=bu, G=out(M, 40, "bf16")[0])
            torch.cuda.synchronize()
            check(X, Wg, Wu, bg, bu, "gelu", H, G, None)


@pytest.mark.parametrize("M,K", [(2, 64), (70, 64), (70, 20000), (300, 512)])
def test_infinities_stay_in_their_rows_and_columns(M, K):  # in each of the forms
    r = np.random.default_rng(933)
    X, Wg, Wu = mat(r, M, K, "f16"), mat(r, 150, K, "f16", 0.1), mat(r, 150, K, "f16", 0.1)
    want, _, _ = rb.qat_glu(X, Wg, Wu, h_dtype=torch.float32)
    X[1, 3], Wg[7, 5], Wu[149, K - 1] = float("inf"), float("nan"), float("-inf")
    H, _, _ = rb.qat_glu(X, Wg, Wu, h_dtype=torch.float32)
    torch.cuda.synchronize()
    keep_r, keep_c = np.delete(np.arange(M), 1), np.delete(np.arange(150), [7, 149])
    assert torch.equal(H[keep_r][:, keep_c], want[keep_r][:, keep_c])
    assert bool(torch.isnan(H[:, 7]).all()) and not bool(torch.isfinite(H[1]).any()) and not bool(torch.isfinite(H[0, 149]))


# ------------------------------------------------------------------------------------------------
# the epilogue's backward
# ------------------------------------------------------------------------------------------------
def check_grad(dH, G, Uu, act, dG, dU, dbg, dbu):
    d, g, u = n64(dH), n64(G), n64(Uu)
    rg, ru, sg, su = BO.glu_backward(d, g, u, act)
    a = BO.activation(g, act)[0]
    lg = (24 * U * (1 + np.abs(g)) * np.abs(u) + 3 * U * np.abs(u)) * np.abs(d) + 3 * U * np.abs(rg)
    lu = 16 * U * (np.abs(g) + np.abs(a)) * np.abs(d) + 2 * U * np.abs(ru)
    near(dG, rg, lg, "dG")
    near(dU, ru, lu, "dU")
    M = d.shape[0]
    if dbg is not None:
        near(dbg, sg, lg.sum(0) + M * U * np.abs(rg).sum(0), "dbg")
    if dbu is not None:
        near(dbu, su, lu.sum(0) + M * U * np.abs(ru).sum(0), "dbu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,ddt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_backward(act, dt, ddt):
    r = np.random.default_rng(940)
    for M, N, pad, off in ((1, 1, 0, 0), (3, 7, 2, 1), (8, 512, 0, 0), (9, 513, 0, 0), (130, 1030, 3, 1), (300, 2048, 8, 8)):
        dH, G, Uu = mat(r, M, N, ddt, 0.1, pad, off), mat(r, M, N, dt, 2.0, pad, off), mat(r, M, N, dt, 1.0, pad, off)
        (dG, bG), (dU, bU) = out(M, N, dt, pad, off), out(M, N, dt, pad, off)
        res = rb.qat_glu_backward(dH, G, Uu, act=act, bias=True, dG=dG, dU=dU)
        torch.cuda.synchronize()
        check_grad(dH, G, Uu, act, *res)
        untouched(dG, bG, M, N, pad, off)
        untouched(dU, bU, M, N, pad, off)


@pytest.mark.parametrize("M,N", [(5, 37), (70, 1031), (200, 1536)])
def test_backward_in_place(M, N):
    """dG and dU over any two of dH, G and U."""
    r = np.random.default_rng(941)
    src = [mat(r, M, N, "bf16", s) for s in (0.1, 2.0, 1.0)]
    want = rb.qat_glu_backward(*src, bias=True)
    for a in range(3):
        for b in range(3):
            if a == b:
                continue
            t = [x.clone() for x in src]
            got = rb.qat_glu_backward(*t, bias=True, dG=t[a], dU=t[b])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want)), (a, b)


def test_backward_with_one_bias_or_none():
    r = np.random.default_rng(942)
    src = [mat(r, 100, 300, "f16", s) for s in (0.1, 2.0, 1.0)]
    full = rb.qat_glu_backward(*src, bias=True)
    buf = torch.empty(300, device=dev())
    for kw in (dict(dbg=buf), dict(dbu=buf), dict()):
        dG, dU, dbg, dbu = rb.qat_glu_backward(*src, **kw)
        torch.cuda.synchronize()
        assert torch.equal(dG, full[0]) and torch.equal(dU, full[1])
        assert (dbg is None) == ("dbg" not in kw) and (dbu is None) == ("dbu" not in kw)
        for a, b in ((dbg, full[2]), (dbu, full[3])):
            assert a is None or torch.equal(a, b)


def test_gradients_at_far_values_are_finite():
    """Slopes are 0 or 1 far out, and a gate of minus many leaves no NaN."""
    g = torch.tensor([[-65504.0, -200.0, -30.0, 30.0, 200.0, 65504.0, 0.0, -0.0]], device=dev(), dtype=torch.float16)
    for act in ACTS:
        dG, dU, _, _ = rb.qat_glu_backward(torch.ones_like(g), g, torch.ones_like(g), act=act)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(dG).all()) and bool(torch.isfinite(dU).all()), act


# ------------------------------------------------------------------------------------------------
# the input's gradient
# ------------------------------------------------------------------------------------------------
def check_dx(dG, dU, Wg, Wu, dX, what="dX"):
    g, u, wg, wu = n64(dG), n64(dU), n64(Wg), n64(Wu)
    S = np.abs(g) @ np.abs(wg) + np.abs(u) @ np.abs(wu)
    near(dX, BO.glu_dx(g, u, wg, wu), (2 * g.shape[1] / 32 + 300) * U * S, what)


def dx_case(seed, M, N, K, dt, xdt=None, pad=0, off=0):
    r = np.random.default_rng([950, seed])
    dG, dU = mat(r, M, N, dt, 0.1, pad, off), mat(r, M, N, dt, 0.1, pad, off)
    Wg, Wu = mat(r, N, K, dt, 0.05, pad, off), mat(r, N, K, dt, 0.05, pad, off)
    dX, buf = out(M, K, xdt or dt, pad, off)
    rb.qat_glu_dx(dG, dU, Wg, Wu, dX=dX)
    torch.cuda.synchronize()
    check_dx(dG, dU, Wg, Wu, dX)
    untouched(dX, buf, M, K, pad, off)


@pytest.mark.parametrize("M", [1, 5, 64, 65, 129, 257])
@pytest.mark.parametrize("N,K", [(8, 8), (64, 64), (72, 256), (136, 264), (1000, 520), (3000, 40)])
def test_dx_edges(M, N, K):
    dx_case(1, M, N, K, "bf16", "f32")


@pytest.mark.parametrize("M", [1, 5, 64, 100, 130])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 5), (7, 64), (63, 9), (65, 257), (997, 300), (64, 250), (66, 256),
                                 (100, 1), (65, 7), (203, 5), (5, 203), (7, 1000)])
def test_dx_edges_unaligned(M, N, K):
    dx_case(2, M, N, K, "f16", "f32")


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (0, 1), (1, 5)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_dx_strides_and_offsets(pad, off, dt):
    for M, N, K in ((1, 40, 200), (40, 264, 72), (150, 1000, 328)):
        dx_case(3, M, N, K, dt, pad=pad, off=off)


@pytest.mark.parametrize("M,N,K", [(512, 512, 1024), (700, 1100, 2048), (2100, 200, 8400), (300, 64, 70000)])
@pytest.mark.parametrize("aligned", [True, False])
def test_dx_many_tiles(M, N, K, aligned):
    r = np.random.default_rng([951, M])
    pad = 0 if aligned else 1
    dG, dU, Wg, Wu = (mat(r, a, b, "bf16", s, pad) for a, b, s in ((M, N, 0.1), (M, N, 0.1), (N, K, 0.05), (N, K, 0.05)))
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu)
    torch.cuda.synchronize()
    at = torch.from_numpy(np.unique(np.r_[0, M - 1, r.integers(0, M, 40)])).to(dev())
    check_dx(dG[at], dU[at], Wg, Wu, dX[at])


@pytest.mark.parametrize("M,N,K", [(3, 24, 40), (70, 1000, 300), (64, 65, 33)])
def test_dx_does_not_read_past_the_sum(M, N, K):
    """Where the sum ends inside a step the elements behind it, here infinite, play no part."""
    r = np.random.default_rng(952)
    full = [mat(r, a, b, "bf16", 0.1) for a, b in ((M, N + 8), (M, N + 8), (N + 8, K + 8), (N + 8, K + 8))]
    dG, dU, Wg, Wu = full[0][:, :N], full[1][:, :N], full[2][:N, :K], full[3][:N, :K]
    want = rb.qat_glu_dx(dG.contiguous(), dU.contiguous(), Wg.contiguous(), Wu.contiguous(), dx_dtype=torch.float32)
    for t in full[:2]:
        t[:, N:] = float("inf")
    for t in full[2:]:
        t[N:] = float("inf")
        t[:, K:] = float("nan")
    got = rb.qat_glu_dx(dG, dU, Wg, Wu, dx_dtype=torch.float32)
    torch.cuda.synchronize()
    check_dx(dG, dU, Wg, Wu, got)
    check_dx(dG, dU, Wg, Wu, want)


# ------------------------------------------------------------------------------------------------
# calls as programs make them
# ------------------------------------------------------------------------------------------------
def everything(seed=7, M=200, N=700, K=1032):
    r = np.random.default_rng([960, seed])
    X, Wg, Wu, dH = mat(r, M, K, "bf16"), mat(r, N, K, "bf16", 0.05), mat(r, N, K, "bf16", 0.05), mat(r, M, N, "bf16", 0.1)

    def go():
        H, G, Uu = rb.qat_glu(X, Wg, Wu, save=True)
        dG, dU, dbg, dbu = rb.qat_glu_backward(dH, G, Uu, bias=True)
        return [H, G, Uu, dG, dU, dbg, dbu, rb.qat_glu_dx(dG, dU, Wg, Wu)]
    return go, (X, Wg, Wu, dH)


def test_equal_calls_give_equal_results_whatever_the_workspace_held():
    r = np.random.default_rng(961)
    X, Wg, Wu = mat(r, 70, 5000, "bf16"), mat(r, 300, 5000, "bf16", 0.05), mat(r, 300, 5000, "bf16", 0.05)
    n = rb.workspace_bytes(rb.RB_OP_QAT_GLU, 1, 300, 5000, 70)  # split tiles
    m = rb.workspace_bytes(rb.RB_OP_QAT_GLU_DX, 1, 300, 5000, 70)
    assert n > 0
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev())
        ws2 = torch.full((max(m, 16),), fill, dtype=torch.uint8, device=dev())
        H, _, _ = rb.qat_glu(X, Wg, Wu, ws=ws)
        dX = rb.qat_glu_dx(H, H, Wg, Wu, ws=ws2)
        torch.cuda.synchronize()
        # the zero region in front of it is never written
        assert bool((ws[:2400 // 256 * 256] == fill).all())
        first = first or (H.clone(), dX.clone())
        assert torch.equal(H, first[0]) and torch.equal(dX, first[1])


def test_captured_and_replayed():
    go, (X, Wg, Wu, dH) = everything()
    go()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = go()
    for k in range(3):
        X.copy_(torch.randn_like(X.float()).to(X.dtype))
        dH.copy_((torch.randn_like(dH.float()) * 0.1).to(dH.dtype))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_two_streams_at_once():
    jobs = [everything(s) for s in (1, 2)]
    want = [go() for go, _ in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [None, None]
    for _ in range(3):
        for i, (go, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i] = go()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_2_32_elements():
    """Weights of 2^22 rows: forward in its rows' and tiles' forms, and the backward's sum over them."""
    N, K = (1 << 22) + 5, 1032
    Wg, Wu = (torch.empty((N, K), dtype=torch.bfloat16, device=dev()).normal_(std=0.03) for _ in range(2))
    cols = torch.tensor([0, 1, 1 << 20, (1 << 22) - 1, 1 << 22, N - 1], device=dev())
    r = np.random.default_rng(970)
    for M in (3, 40):
        X = mat(r, M, K, "bf16")
        H, G, Uu = rb.qat_glu(X, Wg, Wu, save=True)
        torch.cuda.synchronize()
        check(X, Wg[cols], Wu[cols], None, None, "silu", H[:, cols], G[:, cols], Uu[:, cols])
    dG, dU = (torch.zeros((40, N), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    at = torch.tensor([3, 77777, 1 << 21, N - 9, N - 1], device=dev())
    dG[:, at], dU[:, at] = mat(r, 40, 5, "bf16"), mat(r, 40, 5, "bf16")
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu, dx_dtype=torch.float32)
    torch.cuda.synchronize()
    check_dx(dG[:, at], dU[:, at], Wg[at], Wu[at], dX)


def test_outputs_past_2_32_elements():
    M, N = 70, 200
    ld = 1 << 26
    big = torch.empty((M, ld), dtype=torch.bfloat16, device=dev())
    r = np.random.default_rng(971)
    X, Wg, Wu = mat(r, M, 64, "bf16"), mat(r, N, 64, "bf16", 0.1), mat(r, N, 64, "bf16", 0.1)
    H, G, Uu = rb.qat_glu(X, Wg, Wu, H=big[:, :N], G=big[:, 1000:1000 + N], U=big[:, 5000:5000 + N])
    torch.cuda.synchronize()
    check(X, Wg, Wu, None, None, "silu", H, G, Uu)
    dG, dU, dbg, dbu = rb.qat_glu_backward(H, G, Uu, bias=True, dG=big[:, 9000:9000 + N], dU=big[:, 9500:9500 + N])
    torch.cuda.synchronize()
    check_grad(H, G, Uu, "silu", dG, dU, dbg, dbu)
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu, dX=big[:, 20000:20064])
    torch.cuda.synchronize()
    check_dx(dG, dU, Wg, Wu, dX)


def test_weight_gradients_without_an_input_gradient():
    """rb_qat_backward with no dX gives the other three as with one."""
    r = np.random.default_rng(980)
    M, N, K = 100, 72, 136
    W = mat(r, N, K, "f32", 0.1)
    g, h = W.abs().mean(1)[None].contiguous(), torch.ones((1, K), device=dev())
    planes, What = rb.qat_derive(W, g, h, a_dtype=torch.bfloat16)
    X, dY = mat(r, M, K, "bf16"), mat(r, M, N, "bf16")
    full = rb.qat_backward(dY, X, What, planes, g, h)
    part = rb.qat_backward(dY, X, What, planes, g, h, need_dx=False)
    torch.cuda.synchronize()
    assert part[1] is None
    assert all(torch.equal(a, b) for a, b in zip((full[0], *full[2:]), (part[0], *part[2:])))


@pytest.mark.parametrize("M,K", [(5, 8), (16, 9), (12, 64)])
def test_weight_rows_past_one_launch(M, K):
    """2^27 weight rows and more in the one-launch form, 512 threads for every 16: past 2^32 threads. Every output is
    written, sampled ones are right."""
    N = (1 << 27) + 37
    X, Wg, Wu = long_buffer(M, K, DT["bf16"]), long_buffer(N, K, DT["bf16"]), long_buffer(N, K, DT["bf16"])
    bg, bu = long_buffer(1, N, torch.float32)[0], long_buffer(1, N, torch.float32)[0]
    H, G, Uu = (long_buffer(M, N, DT["bf16"], float("nan")) for _ in range(3))
    rb.qat_glu(X, Wg, Wu, bias_g=bg, bias_u=bu, H=H, G=G, U=Uu)
    assert not any(bool(torch.isnan(t).any()) for t in (H, G, Uu))
    for p in pieces(N):
        check(X, Wg[p], Wu[p], bg[p], bu[p], "silu", H[:, p], G[:, p], Uu[:, p])
    del Wg, Wu, H, G, Uu
    torch.cuda.empty_cache()


def test_many_batch_rows():
    """2^24 batch rows and more, each direction: tiles along the batch, strips of many rows."""
    M, N, K = (1 << 24) + 77, 24, 16
    X, Wg, Wu = long_buffer(M, K, DT["bf16"]), long_buffer(N, K, DT["bf16"]), long_buffer(N, K, DT["bf16"])
    H, G, Uu = (long_buffer(M, N, DT["bf16"], float("nan")) for _ in range(3))
    rb.qat_glu(X, Wg, Wu, H=H, G=G, U=Uu)
    assert not any(bool(torch.isnan(t).any()) for t in (H, G, Uu))
    for p in pieces(M):
        check(X[p], Wg, Wu, None, None, "silu", H[p], G[p], Uu[p])
    dH = long_buffer(M, N, DT["bf16"])
    dG, dU, _, _ = rb.qat_glu_backward(dH, G, Uu)
    for p in pieces(M):
        check_grad(dH[p], G[p], Uu[p], "silu", dG[p], dU[p], None, None)
    # sums of M equal terms: 1024 strips, a thread's run of 4097 rows of one, their 1024 sums in 8 runs; a strip's part is 2^-10
    one = torch.ones((M, N), dtype=torch.bfloat16, device=dev())
    _, _, dbg, dbu = rb.qat_glu_backward(one, one, one, bias=True)
    g = 1 / (1 + np.exp(-1.0))
    for got, each in ((dbg, g + g * (1 - g)), (dbu, g)):
        near(got, np.full(N, M * each), (4097 + 3 + 128 + 8 + 24 * 2) * U * M * each, "column sums")
    del one
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu)
    for p in pieces(M):
        check_dx(dG[p], dU[p], Wg, Wu, dX[p])
    del X, H, G, Uu, dH, dG, dU, dX
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [3, 40, 300])
def test_rows_far_apart(M):
    """Leading dimensions of 2^21 and more, aligned: past what a tile's buffer loads reach."""
    N, K, ld = 130, 200, (1 << 21) + 8
    X, Wg, Wu, dG, dU = (long_buffer(n, ld, DT["f16"])[:, :k] for n, k in ((M, K), (N, K), (N, K), (M, N), (M, N)))
    H, G, Uu = rb.qat_glu(X, Wg, Wu, act="gelu", h_dtype=torch.float32, save=True)
    dX = rb.qat_glu_dx(dG, dU, Wg, Wu, dx_dtype=torch.float32)
    torch.cuda.synchronize()
    check(X, Wg, Wu, None, None, "gelu", H, G, Uu)
    check_dx(dG, dU, Wg, Wu, dX)
    del X, Wg, Wu, dG, dU
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K", [(3, (1 << 24) + 5), (70, (1 << 21) + 8), (300, 1 << 21)])
def test_dx_of_many_columns(M, K):
    """dX of 2^21 columns and more, where its weights' rows are past the aligned tiles' reach."""
    N = 24
    dG, dU = long_buffer(M, N, DT["bf16"]), long_buffer(M, N, DT["bf16"])
    Wg, Wu = long_buffer(N, K, DT["bf16"]), long_buffer(N, K, DT["bf16"])
    dX = long_buffer(M, K, DT["bf16"], float("nan"))
    rb.qat_glu_dx(dG, dU, Wg, Wu, dX=dX)
    assert not torch.isnan(dX).any()
    for p in pieces(K):
        check_dx(dG, dU, Wg[:, p], Wu[:, p], dX[:, p])
    del Wg, Wu, dX
    torch.cuda.empty_cache()
