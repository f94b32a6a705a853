"""GPU parity of the layer's product with its epilogue (rb_qat_linear) and of the epilogue's backward
(rb_qat_linear_backward) against the oracle.

Comparison rules, u = 2^-24:
* Z: the products of fp16/bf16 numbers are exact in fp32; they are added 32 to a matrix instruction and
  K / 32 instructions deep, the halves of a step's columns and the K chunks joined after: at most
  (K / 32 + 48) u of S = sum |x w| + |b|, for the K here below 2e-5 S;
* Y: every activation's slope is below 1.13, its own evaluation (exp and erf of the device, a reciprocal)
  within 16 u of |z| + |act(z)|, plus the residual's and the sum's rounding;
* dZ: the slope's evaluation within 24 u (1 + |z|) of |dY|; db: those errors and M u of sum |dZ|;
* rounded outputs add half a unit of their type.
"""
import math

import numpy as np
import pytest
import torch

import residual_binarized_weight_amd as rb
from oracle import block_oracle as BO
from tests import linear_forms as F
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


def near(got, ref, lim, what):
    lim = lim + UNIT[got.dtype] * np.abs(ref) + TINY[got.dtype]
    err = np.abs(n64(got) - ref)
    assert np.all(err <= lim), f"{what}: {np.nanmax(err / lim):.3g} x the bound, {np.isnan(err).sum()} NaN"


def case(seed, M, N, K, dt, act="none", bias=False, res=False, ydt=None, save_z=False, pad=0, off=0):
    r = np.random.default_rng([920, seed])
    ydt = ydt or dt
    X, W = mat(r, M, K, dt, 1.0, pad, off), mat(r, N, K, dt, 0.03, pad, off)
    b = torch.from_numpy(r.standard_normal(N).astype(np.float32)).to(dev()) if bias else None
    R = mat(r, M, N, ydt, 1.0, pad, off) if res else None
    Y, Z = rb.qat_linear(X, W, bias=b, act=act, residual=R, y_dtype=DT[ydt], save_z=save_z)
    torch.cuda.synchronize()
    check(X, W, b, act, R, Y, Z)
    assert (Z is not None) == save_z and Y.dtype == DT[ydt]
    return X, W, b, R, Y, Z


def check(X, W, b, act, R, Y, Z):
    x, w = n64(X), n64(W)
    yo, zo = BO.linear(x, w, n64(b), act, n64(R))
    S = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(n64(b)))
    if Z is not None:
        near(Z, zo, 2e-5 * S, "Z")
    lim = 1.13 * 2e-5 * S + 16 * U * (np.abs(zo) + np.abs(BO.activation(zo, act)[0]))
    near(Y, yo, lim + 2 * U * (np.abs(yo) + (0 if R is None else np.abs(n64(R)))), "Y")


# sizes around every tile edge: 16, 32, 64 and 128 batch rows, 64 and 256 weight rows, 32, 64 and 128 columns
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("N,K", [(1, 8), (63, 64), (256, 72), (257, 128), (300, 136), (65, 1000)])
def test_tile_edges(M, N, K):
    case(1, M, N, K, "bf16", bias=True, ydt="f32")


@pytest.mark.parametrize("M", [1, 3, 16, 31, 64, 100, 130])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (64, 63), (255, 65), (258, 129), (100, 997)])
def test_tile_edges_unaligned(M, N, K):
    case(2, M, N, K, "f16", bias=True, ydt="f32")


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (0, 1), (1, 5)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_strides_and_offsets(pad, off, dt):
    """Rows further apart than their length, with NaN between them, at aligned and odd addresses."""
    for M, K in ((1, 200), (40, 264), (150, 328)):
        case(3, M, 70, K, dt, act="silu", bias=True, res=True, save_z=True, pad=pad, off=off)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("bias,res,save_z", [(False, False, False), (True, True, True), (False, True, False), (True, False, True)])
def test_epilogues(act, dt, ydt, bias, res, save_z):
    case(4, 37, 130, 160, dt, act, bias, res, ydt, save_z)
    case(5, 37, 2050, 2048, dt, act, bias, res, ydt, save_z)      # split columns: the join's epilogue


# the same edges where more rows, or longer ones, bring the tiles
@pytest.mark.parametrize("M", [257, 271, 288, 321, 400])
@pytest.mark.parametrize("N,K", [(1, 8), (63, 64), (257, 72), (300, 136), (65, 1000)])
def test_tile_edges_of_more_rows(M, N, K):
    case(8, M, N, K, "bf16", bias=True, ydt="f32")


@pytest.mark.parametrize("M", [257, 290, 385])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (64, 63), (258, 129), (100, 997)])
def test_tile_edges_unaligned_of_more_rows(M, N, K):
    case(9, M, N, K, "f16", bias=True, ydt="f32")


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (1, 5)])
def test_strides_and_offsets_of_more_rows(pad, off):
    for K in (200, 2056):
        case(10, 300, 70, K, "bf16", act="silu", bias=True, res=True, save_z=True, pad=pad, off=off)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("f16", "f32")])
def test_epilogues_of_more_rows(act, dt, ydt):
    case(11, 290, 130, 160, dt, act, True, True, ydt, True)
    case(12, 60, 1030, 4104, dt, act, True, True, ydt, True)      # split columns: the join's epilogue


@pytest.mark.parametrize("M,N,K", [(20, 1030, 8200), (61, 1027, 1411), (100, 2050, 2056), (129, 3000, 1000), (200, 1500, 2049)])
def test_middle_rows(M, N, K):
    case(13, M, N, K, "bf16", "gelu", True, True, "bf16", True)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 1000, 9000), (17, 520, 8192), (300, 700, 4100), (1100, 4100, 520),
                                   (2048, 4096, 1024), (700, 11008, 640), (7, 4200, 8200)])
def test_long_and_wide(M, N, K):
    case(6, M, N, K, "bf16", "gelu_tanh", True, True, "f32")


@pytest.mark.parametrize("M,N,K", [(1, 2000, 4099), (3, 3000, 2049), (9, 3000, 3001), (40, 1500, 3001), (513, 1030, 1027)])
def test_long_and_wide_unaligned(M, N, K):
    case(7, M, N, K, "f16", "gelu", True, True, "f16", True)


def test_training_shape_sampled():
    """2048 tokens through the 4096 x 11008 layer: sampled rows, first and last included. K = 11008 adds
    (344 + 48) u, still below 2.4e-5: the bound here is 2.4e-5 of S."""
    r = np.random.default_rng(8)
    M, N, K = 2048, 4096, 11008
    X, W = mat(r, M, K, "bf16"), mat(r, N, K, "bf16", 0.03)
    Y, _ = rb.qat_linear(X, W, y_dtype=torch.float32)
    torch.cuda.synchronize()
    rows = [0, 1, 127, 128, 1000, 1531, 2046, 2047]
    x, w = n64(X[rows]), n64(W)
    near(Y[rows], x @ w.T, 2.4e-5 * (np.abs(x) @ np.abs(w).T), "Y")


def test_writes_stay_inside_and_residual_in_place():
    r = np.random.default_rng(9)
    M, N, K = 67, 131, 96
    X, W = mat(r, M, K, "bf16"), mat(r, N, K, "bf16", 0.1)
    Yb, Zb = (torch.full((M + 2, N + 9), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    Y, Z = Yb[1:M + 1, 3:N + 3], Zb[1:M + 1, 5:N + 5]
    R = Y.clone()
    rb.qat_linear(X, W, residual=Y, Y=Y, Z=Z)
    torch.cuda.synchronize()
    check(X, W, None, "none", R, Y, Z)
    for b, o in ((Yb, 3), (Zb, 5)):
        assert torch.all(b[0] == 7) and torch.all(b[M + 1:] == 7) and torch.all(b[:, :o] == 7) and torch.all(b[:, o + N:] == 7)


def test_non_finite_values_stay_in_their_row_and_column():
    r = np.random.default_rng(10)
    X, W = mat(r, 50, 200, "f16"), mat(r, 300, 200, "f16")
    X[7, 3], W[11, 199] = float("nan"), float("inf")
    Y, _ = rb.qat_linear(X, W, y_dtype=torch.float32)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(Y)
    want = torch.zeros_like(bad)
    want[7], want[:, 11] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("M,N,K", [(300, 520, 1600), (3, 4096, 4096), (33, 100, 3001)])
def test_deterministic_and_in_a_graph(M, N, K):
    r = np.random.default_rng(11)
    X, W = mat(r, M, K, "bf16"), mat(r, N, K, "bf16", 0.1)
    want, _ = rb.qat_linear(X, W, y_dtype=torch.float32)
    n = rb.workspace_bytes(rb.RB_OP_QAT_LINEAR, 1, N, K, M)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dev())
    Y = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rb.qat_linear(X, W, Y=Y, ws=ws)
    for _ in range(3):
        ws.fill_(255)
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_on_another_stream():
    r = np.random.default_rng(12)
    X, W = mat(r, 100, 512, "bf16"), mat(r, 600, 512, "bf16", 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Y, Z = rb.qat_linear(X, W, act="silu", save_z=True)
        dZ, db = rb.qat_linear_backward(Y, Z, act="silu")
    s.synchronize()
    check(X, W, None, "silu", None, Y, Z)


# ---------------------------------------------------------------------------------------------
# the epilogue's backward
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 700), (3, 512), (4, 513), (130, 7), (1000, 1030)])
def test_backward(act, dt, ydt, M, N):
    r = np.random.default_rng([921, M, N])
    dY, Z = mat(r, M, N, ydt, 0.1, 3, 1), mat(r, M, N, dt, 2.0, 2, 3)
    dZ, db = rb.qat_linear_backward(dY, Z, act=act)
    torch.cuda.synchronize()
    z, d = n64(Z), n64(dY)
    zo, bo = BO.linear_backward(d, z, act)
    lim = 24 * U * (1 + np.abs(z)) * np.abs(d)
    near(dZ, zo, lim, "dZ")
    near(db, bo, lim.sum(axis=0) + M * U * np.abs(zo).sum(axis=0), "db")


def test_backward_without_bias_or_z_and_in_place():
    r = np.random.default_rng(13)
    dY, Z = mat(r, 60, 200, "bf16"), mat(r, 60, 200, "bf16")
    want, db = rb.qat_linear_backward(dY, Z, act="silu")
    same, none = rb.qat_linear_backward(dY, Z, act="silu", bias=False)
    assert none is None and torch.equal(same, want)
    d = dY.clone()
    rb.qat_linear_backward(d, Z, act="silu", dZ=d, db=db)
    assert torch.equal(d, want)
    f = dY.float()
    dZ, db = rb.qat_linear_backward(f, None, a_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(dZ, f.to(torch.bfloat16))
    near(db, n64(f).sum(axis=0), 60 * U * np.abs(n64(f)).sum(axis=0), "db")


@pytest.mark.parametrize("act", ACTS[2:])
def test_slope_is_the_difference_quotient(act):
    """The slope against central differences of the oracle's activation: truncation h^2 / 6 of a third
    derivative below 4."""
    z = torch.linspace(-9, 9, 4001, device=dev()).to(torch.float16).reshape(1, -1)
    one = torch.ones_like(z, dtype=torch.float32)
    dZ, db = rb.qat_linear_backward(one, z, act=act)
    torch.cuda.synchronize()
    zz, h = n64(z), 1e-4
    diff = (BO.activation(zz + h, act)[0] - BO.activation(zz - h, act)[0]) / (2 * h)
    assert np.max(np.abs(n64(db) - diff[0])) <= h * h + 24 * U * 10 + 1e-10 / h


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_of_huge_values(act):
    """0 and 1 for every finite value far out, also where its square or cube overflows."""
    big = torch.tensor([30.0, 1e4, 1e13, 1.5e19, 2e19, 1e30, 3e38], device=dev())
    z = torch.cat([big, -big]).to(torch.bfloat16).reshape(1, -1)
    dZ, db = rb.qat_linear_backward(torch.ones_like(z), z, act=act)
    torch.cuda.synchronize()
    want = [1.0] * 7 + [0.0] * 7
    # -30: slopes of 1e-11 and less
    assert np.all(np.abs(n64(dZ)[0] - want) <= 1e-10) and np.all(np.abs(n64(db) - want) <= 1e-10)


@pytest.mark.parametrize("act", ACTS)
def test_non_finite_z_in_the_activation_and_its_slope(act):
    """A NaN stays one in the value; its slope is NaN but for relu, whose slope is z > 0, as stated."""
    z = torch.tensor([[float("nan"), float("inf"), -float("inf"), 1.0, 0.0, -0.0, -1.0, 2.0]], device=dev())
    X, W = torch.zeros((1, 8), dtype=torch.float16, device=dev()), torch.zeros((8, 8), dtype=torch.float16, device=dev())
    Y, Z = rb.qat_linear(X, W, bias=z[0], act=act, save_z=True)
    dZ, db = rb.qat_linear_backward(torch.ones_like(Z), Z, act=act)
    torch.cuda.synchronize()
    assert np.array_equal(n64(Z), n64(z), equal_nan=True)
    y, d = n64(Y)[0], n64(dZ)[0]
    assert np.isnan(y[0]) and y[1] == np.inf and np.all(np.isfinite(y[3:])) and np.all(np.isfinite(d[3:]))
    if act == "relu":
        assert y[2] == 0 and d.tolist() == [0, 1, 0, 1, 0, 0, 0, 1] and np.array_equal(n64(db), d)
    elif act == "none":
        assert y[2] == -np.inf and np.all(d == 1)
    else:
        assert np.isnan(d[0])


def tail_terms(act, z):
    """Relative errors of the activations' parts at z, in units of U: those of a rounded argument of the normal tail
    (twice its square, z^2, for two roundings) and of the logistic function (seven roundings and the product with
    log2 e); and 40 for exp, the tail's ratio (up to 32), the reciprocal and the products."""
    if act == "gelu":
        return 40 + 3 * z * z
    return 40 + 9 * np.abs(z if act == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))


@pytest.mark.parametrize("act", ACTS[2:])
def test_activations_keep_their_digits_in_the_tails(act):
    """Every value against itself, not against z: z comes exactly, as the bias of a product of zeros."""
    z = torch.linspace(-9, 9, 3001, device=dev())
    X = torch.zeros((1, 8), dtype=torch.bfloat16, device=dev())
    W = torch.zeros((z.numel(), 8), dtype=torch.bfloat16, device=dev())
    Y, _ = rb.qat_linear(X, W, bias=z, act=act, y_dtype=torch.float32)
    torch.cuda.synchronize()
    zz = n64(z)
    ref = zz * tail_cdf(act, zz)
    near(Y[0], ref, tail_terms(act, zz) * U * np.abs(ref), "Y")


@pytest.mark.parametrize("act", ACTS[2:])
def test_slopes_keep_their_digits_in_the_tails(act):
    """Below zero, against the sum of the slope's terms; db of one row is the slope in fp32."""
    z = torch.linspace(-9, -0.25, 3001, device=dev()).to(torch.float16).reshape(1, -1)
    _, db = rb.qat_linear_backward(torch.ones_like(z, dtype=torch.float32), z, act=act)
    torch.cuda.synchronize()
    zz = n64(z)[0]
    g = tail_cdf(act, zz)
    if act == "gelu":
        second = zz * np.exp(-0.5 * zz * zz) / np.sqrt(2 * np.pi)
    else:
        second = zz * g * (1 - g)
        if act == "gelu_tanh":
            second *= 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * zz * zz)
    near(db, g + second, 2 * tail_terms(act, zz) * U * (g + np.abs(second)), "slope")


def tail_cdf(act, z):
    """What the activation multiplies z by, in 64 bits without cancellation."""
    if act == "gelu":
        return 0.5 * np.vectorize(math.erfc)(-z / math.sqrt(2.0))
    a = z if act == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    return 1 / (1 + np.exp(-a))


def test_refusals():
    r = np.random.default_rng(14)
    X, W = mat(r, 4, 64, "bf16"), mat(r, 8, 64, "bf16")
    with pytest.raises(ValueError):
        rb.qat_linear(X, W[:, :32])
    with pytest.raises(ValueError):
        rb.qat_linear(X, W, bias=torch.zeros(9, device=dev()))
    with pytest.raises(ValueError):
        rb.qat_linear(X, W, residual=torch.zeros((4, 8), device=dev()), Y=torch.zeros((4, 8), dtype=torch.bfloat16, device=dev()))
    with pytest.raises(KeyError):
        rb.qat_linear(X, W, act="tanh")
    with pytest.raises(ValueError):
        rb.qat_linear(X.cpu(), W.cpu())
    with pytest.raises(rb.RbError):
        rb.qat_linear(X.float(), W.float())
    with pytest.raises(rb.RbError):
        rb.qat_linear(X, W, y_dtype=torch.float16)
    with pytest.raises(rb.RbError):
        rb.qat_linear(mat(r, 40, 8192, "bf16"), mat(r, 64, 8192, "bf16"), ws=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(rb.RbError):
        rb.qat_linear_backward(X, None, act="relu", a_dtype=torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# more rows than one launch takes
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 3])
def test_weight_rows_past_one_launch(M):
    """2^26 weight rows and more (2^32 threads), 4.8 G elements apart from first to last: every output is written,
    sampled ones are right."""
    N, K = (1 << 26) + 37, 8
    W = long_buffer(N, 72, DT["bf16"])[:, :K]
    X, b = long_buffer(M, K, DT["bf16"]), long_buffer(1, N, torch.float32)[0]
    R = long_buffer(M, N, torch.float32)
    Y, Z = long_buffer(M, N, torch.float32, float("nan")), long_buffer(M, N, DT["bf16"], float("nan"))
    rb.qat_linear(X, W, bias=b, act="silu", residual=R, Y=Y, Z=Z)
    assert not torch.isnan(Y).any() and not torch.isnan(Z).any()
    for p in pieces(N):
        check(X, W[p], b[p], "silu", R[:, p], Y[:, p], Z[:, p])
    del W, b, R, Y, Z
    torch.cuda.empty_cache()


def test_batch_rows_past_one_launch():
    """2^30 batch rows and more: 2^23 tiles of 512 threads, 8.6 G elements in X and in Y."""
    M, N, K = (1 << 30) + 77, 8, 8
    W, X = long_buffer(N, K, DT["f16"]), long_buffer(M, K, DT["f16"])
    Y = long_buffer(M, N, DT["f16"], float("nan"))
    rb.qat_linear(X, W, act="relu", Y=Y)
    assert not torch.isnan(Y).any()
    for p in pieces(M):
        check(X[p], W, None, "relu", None, Y[p], None)
    del X, Y
    torch.cuda.empty_cache()


def test_backward_offsets_past_32_bits():
    """4.3 G elements a tensor, dZ in place of dY."""
    M, N = (1 << 29) + 77, 8
    dY, Z = long_buffer(M, N, DT["f16"]), long_buffer(M, N, DT["f16"])
    some = [n64(dY[p]) for p in pieces(M)]
    _, db = rb.qat_linear_backward(dY, Z, act="silu", dZ=dY)
    for p, d in zip(pieces(M), some):
        z = n64(Z[p])
        near(dY[p], BO.linear_backward(d, z, "silu")[0], 24 * U * (1 + np.abs(z)) * np.abs(d), "dZ")
    assert torch.isfinite(db).all()
    del dY, Z
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------------------------
# every form of the product: what the tests above ask of some shapes, asked of each
# ---------------------------------------------------------------------------------------------
FORMS = [
    ("rows", 1, 131, 96), ("rows", 3, 131, 97), ("rows", 4, 2051, 96), ("few", 67, 131, 96), ("few", 61, 131, 97),
    ("32", 300, 131, 96), ("32", 300, 131, 97), ("32+join", 300, 131, 2056), ("32+join", 300, 131, 2057),
    ("64", 900, 2050, 72), ("64", 900, 2050, 73), ("64+join", 513, 67, 8200), ("64+join", 513, 67, 2057),
    ("128", 1999, 2050, 72), ("128", 1999, 2050, 73), ("128+join", 1300, 67, 8200), ("128+join", 1300, 67, 2057),
    ("128", 1537, 4100, 515), ("128+join", 1000, 4096, 2050),
    ("256", 1999, 8190, 72), ("256", 4096, 4096, 200), ("256", 257, 32765, 72), ("256+32", 1999, 8203, 72),
    ("256+64", 1537, 11003, 72), ("256+128", 2000, 11003, 1024),
]
TYPES = [("bf16", "f32", "odd"), ("bf16", "bf16", "lines"), ("f16", "f16", "odd"), ("f16", "f32", "lines")]


def form_id(f):
    return f"{f[0]}-{f[1]}x{f[2]}x{f[3]}"


def operands(seed, M, N, K, dt, form):
    assert F.form(M, N, K, K % 8 == 0) == form
    torch.manual_seed(seed)
    return (torch.randn((M, K), device=dev()).to(DT[dt]), torch.randn((N, K), device=dev()).mul_(0.1).to(DT[dt]))


def check_on_gpu(X, W, b, act, R, Y, Z):
    """check() in 64 bits on the GPU, for the large ones."""
    x, w = X.double(), W.double().t().contiguous()
    S = x.abs() @ w.abs() + b.double().abs()
    zo = x @ w + b.double()
    yo = zo * torch.sigmoid(zo) if act == "silu" else zo
    a = yo.abs()
    yo = yo + (0 if R is None else R.double())
    r = 0 if R is None else R.double().abs()
    for got, ref, lim, what in ((Z, zo, 2e-5 * S, "Z"),
                                (Y, yo, 1.13 * 2e-5 * S + 16 * U * (zo.abs() + a) + 2 * U * (yo.abs() + r), "Y")):
        err = (got.double() - ref).abs()
        ok = err <= lim + UNIT[got.dtype] * ref.abs() + TINY[got.dtype]
        assert ok.all(), (what, int((~ok).sum()), (~ok).nonzero()[:3].tolist())


@pytest.mark.parametrize("dt,ydt,place", TYPES)
@pytest.mark.parametrize("form", FORMS, ids=form_id)
def test_every_form(form, dt, ydt, place):
    """Bias, activation, residual and kept Z, the outputs inside buffers of 7: rows at odd places with the residual in
    Y itself, or rows that start 128-byte lines with a residual of its own. Nothing around them is written."""
    name, M, N, K = form
    X, W = operands(15, M, N, K, dt, name)
    b = torch.randn(N, device=dev())
    ld, o = (N + 9, 3) if place == "odd" else ((N + 63) // 64 * 64 + 64, 0)
    Yb, Zb = (torch.full((M + 2, ld), 7.0, dtype=DT[t], device=dev()) for t in (ydt, dt))
    Y, Z = Yb[1:M + 1, o:N + o], Zb[1:M + 1, o:N + o]
    R = torch.randn((M, N), device=dev()).to(DT[ydt])
    if place == "odd":
        Y.copy_(R)
    rb.qat_linear(X, W, bias=b, act="silu", residual=Y if place == "odd" else R, Y=Y, Z=Z)
    torch.cuda.synchronize()
    check_on_gpu(X, W, b, "silu", R, Y, Z)
    for t in (Yb, Zb):
        assert torch.all(t[0] == 7) and torch.all(t[M + 1:] == 7) and torch.all(t[:, :o] == 7) and torch.all(t[:, o + N:] == 7)


@pytest.mark.parametrize("form", [f for f in FORMS if f[1] < 1000 or f[0] in ("256", "256+32")], ids=form_id)
def test_non_finite_values_stay_in_their_row_and_column_in_every_form(form):
    name, M, N, K = form
    X, W = operands(16, M, N, K, "bf16", name)
    m, n = (7 if M > 7 else 0), N - 2
    X[m, 3], W[n, K - 1] = float("nan"), float("inf")
    Y, _ = rb.qat_linear(X, W, y_dtype=torch.float32)
    torch.cuda.synchronize()
    want = torch.zeros((M, N), dtype=torch.bool, device=dev())
    want[m], want[:, n] = True, True
    assert torch.equal(~torch.isfinite(Y), want)


@pytest.mark.parametrize("form", [f for f in FORMS if f[1:] in ((300, 131, 96), (300, 131, 2057), (1999, 8203, 72))], ids=form_id)
def test_tiles_on_another_stream(form):
    name, M, N, K = form
    X, W = operands(17, M, N, K, "f16", name)
    b = torch.zeros(N, device=dev())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Y, Z = rb.qat_linear(X, W, bias=b, act="silu", save_z=True)
    s.synchronize()
    check_on_gpu(X, W, b, "silu", None, Y, Z)
