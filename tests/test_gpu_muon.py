"""GPU parity of the Newton-Schulz step (rb_muon_step) against the oracle, whose X comes from the singular values.

Comparison rules, u = 2^-24:
* the momentum: two roundings of its fp32 arithmetic, 2 u (|m| + |g|);
* X, in the Frobenius norm. Each fp16 rounding is off by 2^-11 at most and 2^-12.2 in the root mean square. Near the
  end an iteration's B X is 2.74 times X (b + c at singular values near 1), so the roundings of B and of X in it are
  each 2.74 * 2^-12.2 = 5.8e-4 of X and that of A |b + 2 c| 2^-12.2 = 1.5e-4; together 8.4e-4 an iteration. Earlier
  ones are carried on with factors near 1 (rotations) or below: over five in quadrature 1.9e-3. The bound is twice
  that, 4e-3, where n is 16 or more and the roundings are many; for smaller n the roundings may all be large and of
  one sign: (2 * 2.74 + 0.71) * 2^-11 = 3e-3 an iteration, with the slope of the polynomial, at most 1.6 in size over
  the values that it maps to (0.68 to 1.21), 3e-3 (1 + 1.6 + .. + 1.6^4) = 4.8e-2;
* W: lr scale times that, and 3 u |W|.
"""
import numpy as np
import pytest
import torch

import residual_binarized_weight_amd as rb
from oracle import block_oracle as BO
from tests.gpu_util import dev

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs the GPU")]

U = 2.0 ** -24


def n64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def mat(r, N, K, dt=torch.float32, std=1.0, pad=0, off=0, rank=0):
    """N rows of K, pad elements between them (NaN) and off before."""
    a = r.standard_normal((N, K)) if not rank else r.standard_normal((N, rank)) @ r.standard_normal((rank, K))
    buf = torch.full((N * (K + pad) + off,), float("nan"), dtype=dt, device=dev())
    v = buf[off:].view(N, K + pad)[:, :K]
    v.copy_(torch.from_numpy((a * std).astype(np.float32)).to(dt).to(dev()))
    return v


def bound(N, K):
    return 4e-3 if min(N, K) >= 16 else 4.8e-2


def fro(a):
    return float(np.linalg.norm(a))


def step(N, K, seed=1, gdt=torch.float32, pad=0, off=0, nesterov=True, gs=None, steps=5, rank=0, std=1e-3, eps=1e-7):
    r = np.random.default_rng([990, seed, N, K])
    W, G = mat(r, N, K, std=0.02, pad=pad, off=off), mat(r, N, K, gdt, std, pad, off, rank)
    m = mat(r, N, K, std=std, pad=pad, off=off, rank=rank)
    O = mat(r, N, K, torch.float16, pad=pad, off=off)
    scale = None if gs is None else torch.tensor([gs], device=dev())
    lr, wd = 0.02, 0.1
    want = BO.muon(n64(W), n64(G), n64(m), lr, 0.95, nesterov, wd, 0.5, steps, eps, 1.0 if gs is None else float(np.float32(gs)))
    m0 = n64(m)
    lim_m = 2 * U * (np.abs(m0) + 2 * np.abs(n64(G)))
    W0 = n64(W)
    rb.muon_step(W, G, m, lr, nesterov=nesterov, weight_decay=wd, scale=0.5, steps=steps, eps=eps, grad_scale=scale, O=O)
    torch.cuda.synchronize()
    assert np.all(np.abs(n64(m) - want[1]) <= lim_m + 2.0 ** -149)
    X = want[2]
    err = fro(n64(O) - X)
    assert err <= (bound(N, K) + 2.0 ** -11) * fro(X) + 2.0 ** -25 * X.size ** 0.5, f"X off by {err / fro(X):.3g}"
    errw = fro(n64(W) - want[0])
    assert errw <= lr * 0.5 * bound(N, K) * fro(X) + 3 * U * fro(W0) + 3 * U * fro(want[0]), f"W off by {errw:.3g}"
    for t in (W, m):  # nothing between the rows is written
        if pad:
            full = t.as_strided((N, K + pad), (K + pad, 1))[:N - 1]
            assert bool(torch.isnan(full[:, K:]).all())


# around the tiles of 256 and the padding to 64, wide, square and tall
@pytest.mark.parametrize("N,K", [(1, 1), (1, 7), (7, 1), (2, 300), (300, 2), (16, 16), (63, 65), (64, 64), (65, 64), (100, 257),
                                 (256, 256), (257, 255), (300, 700), (700, 300), (513, 1030)])
def test_step(N, K):
    step(N, K)


@pytest.mark.parametrize("N,K", [(128, 1000), (200, 2000), (2000, 200), (512, 512), (600, 700), (260, 1500)])
def test_products_of_several_forms(N, K):
    """Sizes at which one step's products take different forms."""
    step(N, K, 6)


@pytest.mark.parametrize("gdt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_types_strides_and_momentum(gdt, pad, off, nesterov):
    for N, K in ((40, 75), (75, 40), (130, 264)):
        step(N, K, 2, gdt, pad, off, nesterov, gs=0.37, std=1.0)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_number_of_products(steps):
    step(48, 96, 3, steps=steps)


@pytest.mark.parametrize("N,K,rank", [(64, 128, 1), (128, 64, 1), (128, 256, 16), (300, 300, 20)])
def test_low_rank(N, K, rank):
    """Where one fp16 for X would be off by up to 15 %."""
    step(N, K, 4, rank=rank)


@pytest.mark.parametrize("std", [1e-12, 1e-6, 1.0, 1e18])
def test_sizes_of_gradients(std):
    """The norm is summed in fp64: squares that leave fp32's range do no harm, and eps decides for the smallest."""
    step(40, 100, 5, std=std, eps=1e-7)
    step(40, 100, 5, std=std, eps=1e-30)


def test_one_entry_above_all_others():
    r = np.random.default_rng(991)
    G = mat(r, 64, 96, std=1e-4)
    G[5, 7] = 50.0
    O = rb.orthogonalize(G, o_dtype=torch.float16)
    torch.cuda.synchronize()
    X = BO.newton_schulz(n64(G))
    assert fro(n64(O) - X) <= (4e-3 + 2.0 ** -11) * fro(X)


@pytest.mark.parametrize("N,K", [(1100, 2600), (2600, 1100), (1500, 1500)])
def test_many_tiles(N, K):
    """Split tiles and their joins; the singular values of the result."""
    r = np.random.default_rng(992)
    G = mat(r, N, K)
    O = rb.orthogonalize(G, o_dtype=torch.float16)
    torch.cuda.synchronize()
    X = G.double()
    X = X / (X.norm() + 1e-7)
    a, b, c = BO.NS_COEFFICIENTS
    X = X.t() if N > K else X
    for _ in range(5):
        A = X @ X.t().contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X.t() if N > K else X
    assert float((O.double() - X).norm()) <= (4e-3 + 2.0 ** -11) * float(X.norm())
    # the same on the transpose, tile for tile: equal to rounding of O
    T = rb.orthogonalize(G.t().contiguous(), o_dtype=torch.float16)
    torch.cuda.synchronize()
    assert torch.equal(T, O.t()) or N == K


def test_long_and_thin():
    r = np.random.default_rng(993)
    G = torch.randn((3, (1 << 21) - 1), device=dev())
    O = rb.orthogonalize(G, o_dtype=torch.float16)
    torch.cuda.synchronize()
    s = torch.linalg.eigvalsh((O.double() @ O.double().t().contiguous()).cpu()).sqrt()
    want = torch.linalg.svdvals(torch.from_numpy(BO.newton_schulz(n64(G)[:, :200000])))
    assert float((s - s.mean()).abs().max()) < 0.1 and 0.6 < float(s.mean()) < 1.25 and want.shape == (3,)


def test_zero_gradient_and_skip():
    r = np.random.default_rng(994)
    W, m = mat(r, 40, 70), torch.zeros((40, 70), device=dev())
    before = W.clone()
    rb.muon_step(W, torch.zeros_like(W), m, 0.5, weight_decay=0.1)
    torch.cuda.synchronize()
    assert torch.equal(W, before * np.float32(1 - 0.05)) and not m.any()
    G, m = mat(r, 40, 70), mat(r, 40, 70)
    keep = [t.clone() for t in (W, m)]
    O = torch.full((40, 70), 5.0, dtype=torch.bfloat16, device=dev())
    rb.muon_step(W, G, m, 0.5, skip=torch.ones(1, dtype=torch.int32, device=dev()), O=O)
    torch.cuda.synchronize()
    assert torch.equal(W, keep[0]) and torch.equal(m, keep[1]) and bool((O == 5).all())
    rb.muon_step(W, G, m, 0.5, skip=torch.zeros(1, dtype=torch.int32, device=dev()), O=O)
    torch.cuda.synchronize()
    assert not torch.equal(W, keep[0]) and not bool((O == 5).any())


def test_a_bad_gradient_makes_it_all_nan():
    r = np.random.default_rng(995)
    for bad in (float("nan"), float("inf")):
        G = mat(r, 30, 50)
        G[3, 4] = bad
        O = rb.orthogonalize(G)
        torch.cuda.synchronize()
        assert bool(torch.isnan(O).all())


def test_without_momentum_or_weights():
    r = np.random.default_rng(996)
    G = mat(r, 90, 64)
    O = rb.orthogonalize(G, o_dtype=torch.float16)
    W = torch.zeros_like(G)
    rb.muon_step(W, G, None, 1.0, scale=1.0)
    torch.cuda.synchronize()
    # W holds -X: O is its rounding
    assert torch.equal((-W).to(torch.float16), O)


def test_equal_steps_give_equal_results_whatever_the_workspace_held():
    r = np.random.default_rng(997)
    G, W0, m0 = mat(r, 300, 600), mat(r, 300, 600), mat(r, 300, 600)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((rb.workspace_bytes(rb.RB_OP_MUON_STEP, 1, 300, 600, 1),), fill, dtype=torch.uint8, device=dev())
        W, m = W0.clone(), m0.clone()
        rb.muon_step(W, G, m, 0.1, ws=ws)
        torch.cuda.synchronize()
        assert bool((ws[:2560 - 160] == fill).all())  # the zero region: 8 bytes a row
        first = first or (W, m)
        assert torch.equal(W, first[0]) and torch.equal(m, first[1])


@pytest.mark.parametrize("N,K", [(200, 456), (1000, 1800)])
def test_captured_and_replayed_beside_another_stream(N, K):
    """In one launch a product, and on tiles with split ones joined."""
    r = np.random.default_rng(998)
    G, W, m = mat(r, N, K), mat(r, N, K), mat(r, N, K)
    other = mat(r, K, N)
    want_other = rb.orthogonalize(other)
    W2, m2 = W.clone(), m.clone()
    rb.muon_step(W.clone(), G, m.clone(), 0.1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rb.muon_step(W, G, m, 0.1)
    side = torch.cuda.Stream()
    for k in range(3):
        G.copy_(torch.randn_like(G))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            got = rb.orthogonalize(other)
        torch.cuda.synchronize()
        rb.muon_step(W2, G, m2, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(W, W2) and torch.equal(m, m2) and torch.equal(got, want_other), k


def columns_near(O, G, axis):
    """O against the products in 64 bits, vector by vector along the long axis: the file's bound for few rows counts every
    rounding at its largest, relative to the vector that it falls on, so that it holds for each of them."""
    X = G.double()
    X = X / (X.norm() + 1e-7)
    a, b, c = BO.NS_COEFFICIENTS
    X = X.t() if axis == 0 else X
    for _ in range(5):
        A = X @ X.t().contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    got = (O.t() if axis == 0 else O).double()
    err, size = (got - X).norm(dim=0), X.norm(dim=0)
    n = X.shape[0]
    assert bool((err <= (bound(*G.shape) + 2.0 ** -11) * size + 2.0 ** -25 * n ** 0.5).all()), f"{float((err / size).max()):.3g}"
    assert float(X.norm()) > 0.6  # its singular values end near 1


@pytest.mark.parametrize("n", [1, 3, 7])
@pytest.mark.parametrize("tall", [False, True])
def test_every_vector_of_long_and_thin_ones(n, tall):
    """Up to the largest length, 2^21 - 1: every column (row) against the definition."""
    m = (1 << 21) - 1
    gen = torch.Generator(device=dev())
    gen.manual_seed(n)
    G = torch.randn((m, n) if tall else (n, m), generator=gen, device=dev())
    O = rb.orthogonalize(G, o_dtype=torch.float16)
    torch.cuda.synchronize()
    columns_near(O, G, 0 if tall else 1)


def test_a_square_matrix_and_its_transpose():
    """Both results are within the bound of one X."""
    G = mat(np.random.default_rng(999), 1500, 1500)
    O, T = (rb.orthogonalize(t, o_dtype=torch.float16) for t in (G, G.t().contiguous()))
    torch.cuda.synchronize()
    size = float(O.double().norm())
    assert float((T.double() - O.t().double()).norm()) <= 2 * (4e-3 + 2.0 ** -11) * size * (1 + 5e-3)
