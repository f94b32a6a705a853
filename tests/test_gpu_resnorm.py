"""GPU parity of the norms between blocks (rb_resnorm_forward / rb_resnorm_backward) against the
oracle, at widths around every change of launch shape, odd ones, strided and unaligned rows.

Comparison rules, u = 2^-24 and D the width: a row's sums are fp32 over at most 16 terms in a thread,
then a tree, so a mean or a mean square is off by at most 24 u of its sum of |terms|, and 1/deviation
by 16 u (relative) plus that of its mean. Values computed from them are bounded by 64 u of the sum
of their |terms| (each factor's relative error added up), plus half a unit of the output's type. The
column sums add M rows of such values: 64 u + M u of the sum of |terms|.
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
EPS = 1e-5


def n64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def mat(r, M, D, dt, std=1.0, ld=None, off=0, mean=0.0):
    """M rows of D, ld elements apart, `off` elements into the buffer; what lies between stays 7."""
    ld = ld or D
    buf = torch.full((M * ld + off,), 7.0, dtype=DT[dt], device=dev())
    v = buf[off:].view(M, ld)[:, :D]
    v.copy_(torch.from_numpy((r.standard_normal((M, D)) * std + mean).astype(np.float32)).to(DT[dt]).to(dev()))
    return v


def vec(r, D, lo=0.5, hi=1.5):
    return torch.from_numpy(r.uniform(lo, hi, D).astype(np.float32)).to(dev())


def near(got, ref, terms, rel, what):
    lim = rel * terms + UNIT[got.dtype] * np.abs(ref) + TINY[got.dtype]
    err = np.abs(n64(got) - ref)
    assert np.all(err <= lim), f"{what}: {np.max(err / lim):.3g} x the bound"


def make(seed, M, D, dt, sdt, post, pre, gate, bias, ld=None, off=0):
    r = np.random.default_rng([910, seed])
    a = dict(Y=mat(r, M, D, dt, 0.7, ld, off, 0.2), R=mat(r, M, D, sdt, 1.0, ld, off), w_pre=vec(r, D), w_post=vec(r, D),
             b_pre=vec(r, D, -1, 1) if bias else None, b_post=vec(r, D, -1, 1) if bias and post != "none" else None,
             gate={"none": lambda: None, "channel": lambda: vec(r, D, -1, 1),
                   "element": lambda: mat(r, M, D, dt, 1.0, ld, off)}[gate](), alpha=0.75, pre=pre, post=post)
    if pre == "none":
        a["w_pre"] = a["b_pre"] = None
    if post == "none":
        a["w_post"] = None
    return a


def ref_args(a):
    return {k: n64(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}


def forward_terms(f):
    """Sums of |terms| of S and X, and the oracle's S, X, stats."""
    S, X, st = BO.resnorm(**f, eps=EPS)
    u = np.abs(f["Y"])
    if f["post"] != "none":
        u = (np.abs(f["Y"]) + np.abs(st[:, 0:1])) * st[:, 1:2] * f["w_post"] + (0 if f["b_post"] is None else np.abs(f["b_post"]))
    if f["gate"] is not None:
        u = np.abs(f["gate"]) * u
    tS = u + (0 if f["R"] is None else f["alpha"] * np.abs(f["R"]))
    tX = None
    if X is not None:
        # an error of S moves the row's statistics as well: by at most its largest term's share of the row
        rms = np.sqrt((tS ** 2).mean(axis=1, keepdims=True))
        tX = (tS + np.abs(st[:, 2:3]) + rms * (1 + np.abs(S) * st[:, 3:4])) * st[:, 3:4] * f["w_pre"]
        tX = tX + (0 if f["b_pre"] is None else np.abs(f["b_pre"]))
    return S, X, st, tS, tX


def check_forward(a, S, X, stats):
    f = ref_args(a)
    So, Xo, sto, tS, tX = forward_terms(f)
    near(S, So, tS, 64 * U, "S")
    if Xo is not None:
        near(X, Xo, tX, 64 * U, "X")
    st = n64(stats)
    scale = np.abs(f["Y"]).mean(axis=1), tS.mean(axis=1)
    for k, kind in ((0, a["post"]), (1, a["pre"])):
        if kind == "none":
            assert np.all(st[:, 2 * k:2 * k + 2] == 0)
            continue
        assert np.all(np.abs(st[:, 2 * k] - sto[:, 2 * k]) <= 64 * U * scale[k])
        # relative to the deviation, S's own errors count by the row's terms
        big = 1 if k == 0 else np.sqrt((tS ** 2).mean(axis=1)) * sto[:, 3]
        assert np.all(np.abs(st[:, 2 * k + 1] / sto[:, 2 * k + 1] - 1) <= 64 * U * np.maximum(1, big))


WIDTHS = [1, 2, 7, 64, 100, 511, 512, 513, 1000, 1024, 1025, 2047, 2049, 4096, 4097, 8191, 8192, 8200, 16384]


@pytest.mark.parametrize("D", WIDTHS)
def test_forward_widths(D):
    for i, (dt, sdt) in enumerate([("bf16", "f32"), ("f16", "f16"), ("f32", "f32")]):
        a = make(i, 5, D, dt, sdt, "layer" if i == 1 else "rms", "rms" if i else "layer", ("channel", "element", "none")[i], True)
        S, X, st = rb.resnorm_forward(**a, eps=EPS)
        torch.cuda.synchronize()
        check_forward(a, S, X, st)


@pytest.mark.parametrize("dt,sdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "none"), ("rms", "rms"), ("layer", "layer"), ("none", "none")])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
def test_forward_kinds(dt, sdt, post, pre, gate):
    a = make(30, 7, 300, dt, sdt, post, pre, gate, gate != "none", ld=311, off=3)
    S, X, st = rb.resnorm_forward(**a, eps=EPS)
    torch.cuda.synchronize()
    assert (X is None) == (pre == "none")
    check_forward(a, S, X, st)


def test_forward_without_residual_and_in_place():
    a = make(40, 33, 520, "f16", "f16", "rms", "rms", "channel", False)
    want = rb.resnorm_forward(**a, eps=EPS)
    Y, R = a["Y"].clone(), a["R"].clone()
    got = rb.resnorm_forward(**{**a, "Y": Y, "R": R}, eps=EPS, S=R, X=Y)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0] is R and got[1] is Y
    b = {**a, "R": None}
    S, X, st = rb.resnorm_forward(**b, eps=EPS)
    torch.cuda.synchronize()
    check_forward(b, S, X, st)


def test_forward_writes_stay_in_the_rows():
    a = make(41, 6, 259, "bf16", "f32", "rms", "rms", "none", False)
    Sb, Xb = torch.full((6, 270), 7.0, device=dev()), torch.full((6, 266), 7.0, dtype=torch.bfloat16, device=dev())
    S, X, st = rb.resnorm_forward(**a, eps=EPS, S=Sb[:, 1:260], X=Xb[:, 3:262])
    torch.cuda.synchronize()
    check_forward(a, S, X, st)
    assert torch.all(Sb[:, 0] == 7) and torch.all(Sb[:, 260:] == 7) and torch.all(Xb[:, :3] == 7) and torch.all(Xb[:, 262:] == 7)


def test_forward_zero_rows_large_means_and_non_finite_rows():
    """A zero row gives zeros (eps holds the division), a mean of 1000 deviations keeps its digits
    (the square of the spread is not a difference), and a NaN stays in its row."""
    r = np.random.default_rng(3)
    Y = torch.from_numpy((r.standard_normal((4, 700)) + 1000).astype(np.float32)).to(dev())
    Y[1] = 0
    Y[2, 5] = float("nan")
    Y[3, 9] = float("inf")
    one = torch.ones(700, device=dev())
    S, X, st = rb.resnorm_forward(Y, None, one, w_post=one, pre="layer", post="layer", eps=EPS)
    torch.cuda.synchronize()
    assert torch.all(S[1] == 0) and torch.all(X[1] == 0)
    assert torch.isnan(X[2]).all() and torch.isnan(S[3]).any()
    ref = BO.norm(n64(Y[:1]), "layer", np.ones(700), None, EPS)
    # the mean, 1000, is off by at most 24 u of itself, against a deviation of 1
    assert np.max(np.abs(n64(S[:1]) - ref)) <= 24 * U * 1000 * 4


def check_backward(a, dX, dS, S, st, got, bias):
    f = ref_args(a)
    g = BO.resnorm_backward(n64(dX), n64(dS), f["Y"], n64(S), n64(st), f["w_pre"], f["w_post"], f["b_post"], f["gate"],
                            f["alpha"], a["pre"], a["post"])
    M, D = f["Y"].shape
    sd = n64(st)
    # |terms| of T: the direct gradient, the norm's own and the row means
    tT = np.zeros((M, D)) if dS is None else np.abs(n64(dS))
    if a["pre"] != "none":
        d, xh = np.abs(n64(dX)) * f["w_pre"], (np.abs(n64(S)) + np.abs(sd[:, 2:3])) * sd[:, 3:4]
        tT = tT + (d + d.mean(axis=1, keepdims=True) + xh * (d * xh).mean(axis=1, keepdims=True)) * sd[:, 3:4]
        near(got["dw_pre"], g["dw_pre"], (np.abs(n64(dX)) * xh).sum(axis=0), (64 + M) * U, "dw_pre")
        if bias:
            near(got["db_pre"], g["db_pre"], np.abs(n64(dX)).sum(axis=0), (64 + M) * U, "db_pre")
    near(got["dR"], g["dR"], f["alpha"] * tT, 64 * U, "dR")
    yh = np.abs(f["Y"])
    if a["post"] != "none":
        yh = (yh + np.abs(sd[:, 0:1])) * sd[:, 1:2]
    tdu = tT
    if f["gate"] is not None:
        u = yh if a["post"] == "none" else yh * f["w_post"] + (0 if f["b_post"] is None else np.abs(f["b_post"]))
        if f["gate"].ndim == 1:
            near(got["dgate"], g["dgate"], (u * tT).sum(axis=0), (64 + M) * U, "dgate")
        else:
            near(got["dgate"], g["dgate"], u * tT, 64 * U, "dgate")
        tdu = np.abs(f["gate"]) * tT
    else:
        assert got["dgate"] is None
    tY = tdu
    if a["post"] != "none":
        e = tdu * f["w_post"]
        tY = (e + e.mean(axis=1, keepdims=True) + yh * (e * yh).mean(axis=1, keepdims=True)) * sd[:, 1:2]
        near(got["dw_post"], g["dw_post"], (tdu * yh).sum(axis=0), (64 + M) * U, "dw_post")
        if bias:
            near(got["db_post"], g["db_post"], tdu.sum(axis=0), (64 + M) * U, "db_post")
    near(got["dY"], g["dY"], tY, 128 * U, "dY")
    for k, there in (("dw_pre", a["pre"] != "none"), ("db_pre", bias and a["pre"] != "none"),
                     ("dw_post", a["post"] != "none"), ("db_post", bias and a["post"] != "none")):
        assert (got[k] is not None) == there


def run_backward(seed, M, D, dt, sdt, post, pre, gate, bias, ld=None, off=0, with_ds=True):
    a = make(seed, M, D, dt, sdt, post, pre, gate, bias, ld, off)
    S, X, st = rb.resnorm_forward(**a, eps=EPS)
    r = np.random.default_rng([911, seed])
    dX = mat(r, M, D, dt, 0.1, ld, off) if pre != "none" else None
    dS = mat(r, M, D, sdt, 0.1, ld, off) if with_ds or pre == "none" else None
    got = rb.resnorm_backward(dX, dS, a["Y"], S, st, a["w_pre"], w_post=a["w_post"], b_post=a["b_post"], gate=a["gate"],
                              alpha=a["alpha"], pre=pre, post=post, bias=bias)
    torch.cuda.synchronize()
    check_backward(a, dX, dS, S, st, got, bias)
    return a, dX, dS, S, st, got


@pytest.mark.parametrize("D", WIDTHS)
def test_backward_widths(D):
    for i, (dt, sdt) in enumerate([("bf16", "f32"), ("f16", "f16"), ("f32", "f32")]):
        run_backward(50 + i, 5, D, dt, sdt, "layer" if i == 1 else "rms", "rms" if i else "layer",
                     ("channel", "element", "none")[i], bool(i))


@pytest.mark.parametrize("dt,sdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "none"), ("rms", "rms"), ("layer", "layer"), ("none", "none")])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
def test_backward_kinds(dt, sdt, post, pre, gate):
    run_backward(70, 7, 300, dt, sdt, post, pre, gate, gate == "element", ld=311, off=3, with_ds=gate != "none")


@pytest.mark.parametrize("M", [1, 3, 255, 256, 257, 600, 2049])
@pytest.mark.parametrize("D", [96, 1030, 2500])
def test_backward_rows(M, D):
    """Row counts around one block each, one round of the blocks' row groups, and several rounds."""
    run_backward(80, M, D, "bf16", "f32", "rms", "rms", "channel", False)


@pytest.mark.parametrize("M", [1, 65, 260, 301])
@pytest.mark.parametrize("D", [8193, 8705, 9001])
def test_backward_wide_rows(M, D):
    """Rows that no block holds: strips of 4 and 5 rows, a last strip with fewer, last columns of 1 to 7."""
    run_backward(100, M, D, "bf16", "bf16", "layer", "layer", "channel", True)


@pytest.mark.parametrize("dt,sdt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "none"), ("layer", "rms"), ("none", "none")])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
def test_backward_wide_kinds(dt, sdt, post, pre, gate):
    run_backward(101, 6, 8300, dt, sdt, post, pre, gate, gate == "element", ld=8311, off=3, with_ds=gate != "none")


@pytest.mark.parametrize("D", [300, 6000, 8300])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_vectors_of_an_absent_norm_are_not_used(D, gate):
    """post "none" with a w_post and a b_post: u is Y itself, in both directions."""
    a, dX, dS, S, st, got = run_backward(103, 6, D, "bf16", "f32", "none", "rms", gate, False)
    r = np.random.default_rng(104)
    w, b = vec(r, D), vec(r, D)
    same = rb.resnorm_forward(**{**a, "w_post": w, "b_post": b}, eps=EPS)
    back = rb.resnorm_backward(dX, dS, a["Y"], S, st, a["w_pre"], w_post=w, b_post=b, gate=a["gate"], alpha=a["alpha"],
                               pre="rms", post="none")
    torch.cuda.synchronize()
    assert torch.equal(same[0], S) and torch.equal(same[2], st)
    assert all(torch.equal(back[k], got[k]) for k in got if got[k] is not None)


def test_backward_wide_in_place_and_deterministic():
    a, dX, dS, S, st, got = run_backward(102, 70, 8705, "bf16", "bf16", "rms", "layer", "channel", False)
    kw = dict(w_post=a["w_post"], gate=a["gate"], alpha=a["alpha"], pre="layer", post="rms")
    for out in ("Y", "dX"):
        x, y, s = dX.clone(), a["Y"].clone(), dS.clone()
        again = rb.resnorm_backward(x, s, y, S, st, a["w_pre"], dY=y if out == "Y" else x, dR=s, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(again[k], got[k]) for k in got if got[k] is not None)


def test_backward_against_differences():
    """Central differences of L = <X, dX> + <S, dS> in the library's own fp32 forward, along random
    directions of every input: their truncation error is h^2 and their rounding 1e-6 / h of |L|'s terms."""
    M, D, h = 3, 130, 2e-2
    a = make(90, M, D, "f32", "f32", "layer", "layer", "channel", True)
    S, X, st = rb.resnorm_forward(**a, eps=EPS)
    r = np.random.default_rng(91)
    dX, dS = mat(r, M, D, "f32"), mat(r, M, D, "f32")
    got = rb.resnorm_backward(dX, dS, a["Y"], S, st, a["w_pre"], w_post=a["w_post"], b_post=a["b_post"], gate=a["gate"],
                              alpha=a["alpha"], pre="layer", post="layer", bias=True)

    def loss(b):
        s, x, _ = rb.resnorm_forward(**b, eps=EPS)
        return float((x.double() * dX.double()).sum() + (s.double() * dS.double()).sum())
    names = dict(Y="dY", R="dR", w_pre="dw_pre", w_post="dw_post", b_pre="db_pre", b_post="db_post", gate="dgate")
    for k, gk in names.items():
        v = torch.from_numpy(r.standard_normal(a[k].shape).astype(np.float32)).to(dev())
        v = v / v.norm()
        diff = (loss({**a, k: a[k] + h * v}) - loss({**a, k: a[k] - h * v})) / (2 * h)
        want = float((got[gk].double() * v.double()).sum())
        assert abs(diff - want) <= 2e-3 * max(1.0, float(got[gk].double().norm())), (k, diff, want)


def test_backward_in_place_and_deterministic():
    a, dX, dS, S, st, got = run_backward(95, 600, 512, "bf16", "bf16", "rms", "rms", "channel", False)
    kw = dict(w_post=a["w_post"], gate=a["gate"], alpha=a["alpha"], pre="rms", post="rms")
    x, s = dX.clone(), dS.clone()
    again = rb.resnorm_backward(x, s, a["Y"], S, st, a["w_pre"], dY=x, dR=s, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(again[k], got[k]) for k in got if got[k] is not None)


def test_graph_replays_give_the_eager_result():
    a, dX, dS, S, st, got = run_backward(96, 300, 1024, "bf16", "f32", "rms", "rms", "channel", False)
    kw = dict(w_post=a["w_post"], gate=a["gate"], alpha=a["alpha"], pre="rms", post="rms")
    ws = torch.empty(rb.workspace_bytes(rb.RB_OP_RESNORM_BACKWARD, 1, 1024, 1, 300), dtype=torch.uint8, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S2, X2, st2 = rb.resnorm_forward(**a, eps=EPS)
        out = rb.resnorm_backward(dX, dS, a["Y"], S2, st2, a["w_pre"], ws=ws, **kw)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(S2, S) and all(torch.equal(out[k], got[k]) for k in got if got[k] is not None)


def test_refusals():
    a = make(97, 4, 64, "bf16", "f32", "rms", "rms", "none", False)
    with pytest.raises(ValueError):
        rb.resnorm_forward(**{**a, "w_pre": a["w_pre"][:32]})
    with pytest.raises(ValueError):
        rb.resnorm_forward(**{**a, "R": a["R"][:2]})
    with pytest.raises(ValueError):
        rb.resnorm_forward(**{**a, "Y": a["Y"].t().contiguous().t()})
    with pytest.raises(KeyError):
        rb.resnorm_forward(**{**a, "pre": "batch"})
    with pytest.raises(rb.RbError):
        rb.resnorm_forward(**a, eps=0.0)
    with pytest.raises(rb.RbError):
        rb.resnorm_forward(**{**a, "w_pre": None})
    wide = torch.zeros((1, 16385), device=dev())
    with pytest.raises(rb.RbError):
        rb.resnorm_forward(wide, None, torch.ones(16385, device=dev()))
    S, X, st = rb.resnorm_forward(**a)
    with pytest.raises(rb.RbError):
        rb.resnorm_backward(None, None, a["Y"], S, st, a["w_pre"], w_post=a["w_post"])


# ---------------------------------------------------------------------------------------------
# more rows than one launch takes
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M,D,ld", [((1 << 26) + 9, 8, 72), ((1 << 20) + 5, 1030, 1040)])
def test_forward_rows_past_one_launch(M, D, ld):
    """2^32 threads and more, and offsets past 2^32 elements: every row is written, and sampled runs of rows are
    what a call on them alone gives (a row's result does not depend on the others)."""
    r = np.random.default_rng(98)
    a = dict(w_pre=vec(r, D), w_post=vec(r, D), gate=vec(r, D), alpha=0.75, pre="rms", post="rms", eps=EPS)
    Y, S, X = long_buffer(M, ld, DT["f16"])[:, :D], long_buffer(M, ld, DT["f16"])[:, :D], long_buffer(M, ld, DT["f16"], float("nan"))[:, :D]
    R = [S[p].clone() for p in pieces(M)]
    _, _, st = rb.resnorm_forward(Y, S, S=S, X=X, **a)
    assert not torch.isnan(X).any() and torch.all(st[:, 1] > 0) and torch.all(st[:, 3] > 0)
    for p, rows in zip(pieces(M), R):
        s, x, t = rb.resnorm_forward(Y[p], rows, **a)
        assert torch.equal(S[p], s) and torch.equal(X[p], x) and torch.equal(st[p], t)
        check_forward({"Y": Y[p], "R": rows, "b_pre": None, "b_post": None, **{k: a[k] for k in a if k != "eps"}}, s, x, t)
    del Y, S, X, st
    torch.cuda.empty_cache()


def test_backward_wide_rows_past_one_launch():
    """The same of the row means' launch: 2^20 rows and more of over 8192 columns, 8.6 G elements a tensor."""
    M, D = (1 << 20) + 3, 8200
    dX, S = long_buffer(M, D, DT["f16"]), long_buffer(M, D, DT["f16"])
    w = vec(np.random.default_rng(99), D)
    st = torch.zeros((M, 4), device=dev())
    st[:, 3] = 1.0
    some = [(dX[p].clone(), S[p].clone()) for p in pieces(M)]
    got = rb.resnorm_backward(dX, None, S, S, st, w, dY=dX)
    for p, (x, s) in zip(pieces(M), some):
        want = rb.resnorm_backward(x, None, s, s, st[p], w)
        assert torch.equal(got["dY"][p], want["dY"]) and torch.equal(got["dR"][p], want["dR"])
    assert torch.isfinite(got["dw_pre"]).all()
    del dX, S, got
    torch.cuda.empty_cache()


def test_backward_offsets_past_32_bits():
    """Rows up to 8192 columns, walked by 256 blocks: 4.3 G elements a tensor, in place."""
    M, D = (1 << 22) + 7, 1030
    dX, S = long_buffer(M, D, DT["f16"]), long_buffer(M, D, DT["f16"])
    w = vec(np.random.default_rng(105), D)
    st = torch.zeros((M, 4), device=dev())
    st[:, 3] = 1.0
    some = [(dX[p].clone(), S[p].clone()) for p in pieces(M)]
    got = rb.resnorm_backward(dX, None, S, S, st, w, dY=dX)
    for p, (x, s) in zip(pieces(M), some):
        want = rb.resnorm_backward(x, None, s, s, st[p], w)
        assert torch.equal(got["dY"][p], want["dY"]) and torch.equal(got["dR"][p], want["dR"])
    assert torch.isfinite(got["dw_pre"]).all()
    del dX, S, got
    torch.cuda.empty_cache()
