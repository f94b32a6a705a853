"""GPU parity of the 4-bit weights (rb_q4_pack, rb_q4_dequant, rb_q4_gemv, rb_q4_glu) against the oracle.

Comparison rules, u = 2^-24:
* packing: codes and scales equal bit for bit (every step of the definition is one fp32 operation);
* reading back: s (q - 8) is exact in fp32, s q + z rounded once: u, and half a unit of the output's type;
* the product adds x (16 + q), at most 31 |x|, in fp32, 32 to a matrix instruction and up to K / 32 + 8 deep, scales the
  sums of a group and takes 24 s (or 16 s - z) times the sum of x off: within (K / 32 + 40) u of
  sum |x| (55 s + |z|);
* the pair: as for the gated block, from those bounds.
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
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def n64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def rows(a, dt, pad=0, off=0):
    """The rows of a, pad elements between them and off before; what lies between is NaN."""
    M, N = a.shape
    buf = torch.full((M * (N + pad) + off,), float("nan"), dtype=DT[dt], device=dev())
    v = buf[off:].view(M, N + pad)[:, :N]
    v.copy_(torch.from_numpy(a.astype(np.float32)).to(DT[dt]).to(dev()))
    return v


def near(got, ref, lim, what):
    lim = lim + UNIT[got.dtype] * np.abs(ref) + TINY[got.dtype]
    err = np.abs(n64(got) - ref)
    assert np.all(err <= lim), f"{what}: {np.nanmax(err / lim):.3g} x the bound, {np.isnan(err).sum()} NaN"


def weights(r, N, K):
    w = r.standard_normal((N, K)) * 0.02 * r.uniform(0.3, 2, (N, 1))
    w[r.random((N, K)) < 0.002] *= 20
    return w


def packed(q, s, z):
    """The oracle's codes and scales as device tensors in the library's layout."""
    dv = lambda a: None if a is None else torch.from_numpy(a).to(dev())  # noqa: E731
    return dv(BO.q4_codes(q).view(np.int32)), dv(s), dv(z)


def random_weight(r, N, K, group, offset):
    q = r.integers(0, 16, (N, K))
    g = -(-K // group)
    s = (r.uniform(0.2, 1, (g, N)) * 0.01).astype(np.float16)
    z = (r.standard_normal((g, N)) * 0.05).astype(np.float16) if offset else None
    return q, s, z


@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (15, 32), (16, 33), (17, 127), (31, 128), (33, 129), (40, 1000), (130, 263)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_pack_and_read_back(N, K, group, offset, dt):
    r = np.random.default_rng([1000, N, K])
    W = rows(weights(r, N, K), dt, *((5, 3) if N % 2 else (0, 0)))
    codes, s, z = rb.q4_pack(W, group=group, offset=offset)
    q, so, zo = BO.q4_quantise(W.float().cpu().numpy(), group, offset)
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), so) and (z is None) == (not offset)
    assert z is None or np.array_equal(z.cpu().numpy(), zo)
    assert np.array_equal(codes.cpu().numpy().view(np.uint32), BO.q4_codes(q))
    ref = BO.q4_values(q, so, zo, group)
    for out, pad in (("f32", 0), ("f16", 3), ("bf16", 8)):
        buf = torch.full((N, K + pad), 77.0, dtype=DT[out], device=dev())
        rb.q4_dequant(codes, s, z, N, K, group=group, What=buf[:, :K])
        torch.cuda.synchronize()
        near(buf[:, :K], ref, U * np.abs(ref), "What")
        assert bool((buf[:, K:] == 77).all())


def test_pack_ties_zeros_and_equal_values():
    w = np.zeros((4, 64))
    w[0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5]     # scale 1: ties to even
    w[1] = 3.0                                              # one value: offset exact, no scale
    w[2, 5] = 1e-7                                          # its scale underflows fp16: all codes zero
    W = rows(w, "f32")
    for offset in (False, True):
        codes, s, z = rb.q4_pack(W, group=32, offset=offset)
        q, so, zo = BO.q4_quantise(w, 32, offset)
        torch.cuda.synchronize()
        assert np.array_equal(codes.cpu().numpy().view(np.uint32), BO.q4_codes(q)) and np.array_equal(s.cpu().numpy(), so)
    assert bool((rb.q4_dequant(codes, s, z, 4, 64, group=32, dtype=torch.float32)[1] == 3).all())


def test_pack_reports_what_it_cannot_hold():
    W = rows(np.ones((20, 200)), "f32")
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    rb.q4_pack(W, d_status=st)
    assert st.item() == 0
    for bad in (float("nan"), float("inf"), -float("inf"), 1e6):
        for offset in (False, True):
            V = W.clone()
            V[19, 199] = bad
            st.fill_(4)
            codes, s, z = rb.q4_pack(V, group=64, offset=offset, d_status=st)
            assert st.item() == 5, (bad, offset)
            back = rb.q4_dequant(codes, s, z, 20, 200, group=64, dtype=torch.float32)
            assert torch.allclose(back[:19], W[:19], rtol=1e-3)      # other groups are as they were


def product_bound(x, s, z, group, K):
    at = np.arange(K) // group
    each = 55 * s.astype(np.float64)[at] + (0 if z is None else np.abs(z.astype(np.float64)[at]))
    return (K / 32 + 40) * U * (np.abs(x) @ each)


def gemv_case(seed, M, N, K, group, offset, dt, ydt=None, pad=0, off=0):
    r = np.random.default_rng([1010, seed, N, K])
    q, s, z = random_weight(r, N, K, group, offset)
    codes, sd, zd = packed(q, s, z)
    x = rows(r.standard_normal((M, K)), dt, pad, off)
    buf = torch.full((M, N + pad), 77.0, dtype=DT[ydt or dt], device=dev())
    rb.q4_gemv(codes, sd, zd, x, N, group=group, y=buf[:, :N])
    torch.cuda.synchronize()
    near(buf[:, :N], n64(x) @ BO.q4_values(q, s, z, group).T, product_bound(n64(x), s, z, group, K), "y")
    assert bool((buf[:, N:] == 77).all())


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 15, 16])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 7), (16, 128), (17, 129), (100, 1000), (33, 4111)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gemv(M, N, K, dt):
    for group in (32, 64, 128):
        gemv_case(1, M, N, K, group, False, dt, "f32")
        gemv_case(2, M, N, K, group, True, dt)


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (0, 1), (1, 5)])
def test_gemv_strides(pad, off):
    for M, K in ((1, 200), (7, 1032), (16, 2051)):
        gemv_case(3, M, 70, K, 64, True, "bf16", pad=pad, off=off)


@pytest.mark.parametrize("N,K", [(4096, 1024), (1030, 11008), (8200, 520)])
@pytest.mark.parametrize("M", [1, 4, 16])
def test_gemv_layers(M, N, K):
    gemv_case(4, M, N, K, 128, False, "f16", "f32")
    gemv_case(5, M, N, K, 32, True, "bf16", "f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,ydt", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_pair(act, dt, ydt):
    for M, N, K, group, og, ou in ((1, 16, 128, 128, False, False), (3, 130, 777, 32, True, True), (16, 45, 3000, 64, False, True),
                                   (2, 4100, 256, 128, True, False)):
        r = np.random.default_rng([1020, N])
        g, u = random_weight(r, N, K, group, og), random_weight(r, N, K, group, ou)
        x = rows(r.standard_normal((M, K)), dt, 3 if M == 3 else 0)
        y = rb.q4_glu(packed(*g), packed(*u), x, N, group=group, act=act, y_dtype=DT[ydt])
        torch.cuda.synchronize()
        xs = n64(x)
        G, V = xs @ BO.q4_values(*g, group).T, xs @ BO.q4_values(*u, group).T
        lg, lu = product_bound(xs, g[1], g[2], group, K), product_bound(xs, u[1], u[2], group, K)
        a = BO.activation(G, act)[0]
        la = 1.13 * lg + 16 * U * (np.abs(G) + np.abs(a))
        near(y, a * V, la * (np.abs(V) + lu) + np.abs(a) * lu + 2 * U * np.abs(a * V), "y")


def test_a_bad_row_of_x_stays_alone():
    r = np.random.default_rng(1030)
    q, s, z = random_weight(r, 50, 300, 64, False)
    w = packed(q, s, z)
    x = rows(r.standard_normal((5, 300)), "f16")
    want = rb.q4_gemv(*w, x, 50, group=64)
    x[2, 17] = float("nan")
    got = rb.q4_gemv(*w, x, 50, group=64)
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[2]).all())
    keep = [0, 1, 3, 4]
    assert torch.equal(got[keep], want[keep])


def test_rows_do_not_depend_on_the_batch():
    r = np.random.default_rng(1031)
    w = packed(*random_weight(r, 300, 1300, 128, True))
    x = rows(r.standard_normal((16, 1300)), "bf16")
    all16 = rb.q4_gemv(*w, x, 300, y_dtype=torch.float32)
    for m in (1, 2, 7):
        got = rb.q4_gemv(*w, x[:m], 300, y_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(got, all16[:m])


def test_offsets_past_2_32_codes():
    """2^22 rows by 2^11 columns: 2^33 codes, read past 2^32."""
    N, K = (1 << 22) + 5, 2048
    tiles = -(-N // 16)
    codes = torch.randint(-(1 << 31), (1 << 31) - 1, (tiles, K // 128, 64, 4), dtype=torch.int32, device=dev())
    s = torch.rand((K // 32, N), device=dev()).mul_(0.01).half()
    x = torch.randn((3, K), device=dev()).half()
    y = rb.q4_gemv(codes, s, None, x, N, group=32, y_dtype=torch.float32)
    What = rb.q4_dequant(codes, s, None, N, K, group=32)
    torch.cuda.synchronize()
    for n in (0, 17, 1 << 21, (1 << 22) - 1, 1 << 22, N - 1):
        w = codes[n // 16].cpu().numpy().view(np.uint32)
        c = np.arange(K)
        q = w[c // 128, 16 * (c % 32 // 8) + n % 16, c % 128 // 32] >> (16 * (c % 2) + 4 * (c % 8 // 2)).astype(np.uint32) & 15
        ref = BO.q4_values(q[None].astype(np.int64), s[:, n:n + 1].cpu().numpy(), None, 32)
        near(What[n:n + 1], ref, 0, "What")
        near(y[:, n:n + 1], n64(x) @ ref.T, product_bound(n64(x), s[:, n:n + 1].cpu().numpy(), None, 32, K), "y")
    codes2, s2, _ = rb.q4_pack(What, group=32)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1 << 21, N - 1], device=dev())
    q, so, _ = BO.q4_quantise(What[at].float().cpu().numpy(), 32, False)
    assert np.array_equal(s2[:, at].cpu().numpy(), so)
    for i, n in enumerate(at.tolist()):
        tile, lanes = BO.q4_codes(q[i:i + 1])[0][:, ::16], codes2[n // 16].cpu().numpy().view(np.uint32)[:, n % 16::16]
        assert np.array_equal(lanes, tile)


def test_captured_and_replayed():
    r = np.random.default_rng(1040)
    W = rows(weights(r, 200, 900), "f32")
    x = rows(r.standard_normal((4, 900)), "f16")

    def go():
        w = rb.q4_pack(W, group=64, offset=True)
        return [*w, rb.q4_gemv(*w, x, 200, group=64), rb.q4_glu(w, w, x, 200, group=64), rb.q4_dequant(*w, 200, 900, group=64)]
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = go()
    for _ in range(3):
        W.copy_(torch.randn_like(W))
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------------------------------------
# every form of the product: 1, 4 and 16 rows, blocks of 16 waves and (above 4096 weight rows, up to 4 rows) of 8, and
# columns in one or several chunks of the loop
# ------------------------------------------------------------------------------------------------
def device_weight(gen, N, K, group, offset):
    """Codes [N][K], and (codes, s, z) as the library takes them, made on the device."""
    q = torch.randint(0, 16, (N, K), generator=gen, device=dev())
    tn, tk = -(-N // 16), -(-K // 128)
    full = torch.zeros((tn * 16, tk * 128), dtype=torch.int64, device=dev())
    full[:N, :K] = q
    t = full.view(tn, 16, tk, 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 6, 5)  # tiles, lane / 16, row, word, column % 2, column / 2
    w = (t << (4 * torch.arange(8, device=dev()).view(2, 4))).sum((-1, -2))
    g = -(-K // group)
    s = (torch.rand((g, N), generator=gen, device=dev()) * 0.8 + 0.2).mul_(0.01).half()
    z = torch.randn((g, N), generator=gen, device=dev()).mul_(0.05).half() if offset else None
    return q, (torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).reshape(tn, tk, 64, 4).contiguous(), s, z)


def some_rows(N):
    return np.unique(np.clip(np.r_[0:20, N // 2:N // 2 + 20, 4080:4120, N - 20:N], 0, N - 1))


def of_rows(q, w, at):
    """Codes, s and z of some weight rows, on the host."""
    i = torch.from_numpy(at).to(dev())
    return q[i].cpu().numpy(), *(None if t is None else t[:, i].cpu().numpy() for t in w[1:])


def form_case(M, N, K, group, offset, dt, pair, act="silu", ydt="f32"):
    gen = torch.Generator(device=dev())
    gen.manual_seed(M * 1000003 + N * 1009 + K)
    x = rows(np.random.default_rng([1050, M, K]).standard_normal((M, K)), dt)
    ws = [device_weight(gen, N, K, group, o) for o in ((offset, not offset) if pair else (offset,))]
    y = torch.full((M, N), float("nan"), dtype=DT[ydt], device=dev())
    if pair:
        rb.q4_glu(ws[0][1], ws[1][1], x, N, group=group, act=act, y=y)
    else:
        rb.q4_gemv(*ws[0][1], x, N, group=group, y=y)
    torch.cuda.synchronize()
    assert not torch.isnan(y).any()
    at, xs = some_rows(N), n64(x)
    got = y[:, torch.from_numpy(at).to(dev())]
    host = [of_rows(*w, at) for w in ws]
    G = [xs @ BO.q4_values(*h, group).T for h in host]
    L = [product_bound(xs, h[1], h[2], group, K) for h in host]
    if not pair:
        near(got, G[0], L[0], "y")
        return
    a = BO.activation(G[0], act)[0]
    la = 1.13 * L[0] + 16 * U * (np.abs(G[0]) + np.abs(a))
    near(got, a * G[1], la * (np.abs(G[1]) + L[1]) + np.abs(a) * L[1] + 2 * U * np.abs(a * G[1]), "y")


def test_device_codes_are_the_oracles():
    gen = torch.Generator(device=dev())
    gen.manual_seed(1)
    q, (codes, _, _) = device_weight(gen, 37, 300, 64, False)
    assert np.array_equal(codes.cpu().numpy().view(np.uint32), BO.q4_codes(q.cpu().numpy()))


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 4, 11, 16])
def test_every_form(M, dt, group, pair):
    for N in (70, 4096, 4100):
        form_case(M, N, 515, group, N == 70, dt, pair, ydt="f32" if N != 4100 else dt)


# a chunk holds 12288 columns (16 waves) or 8192 (8), of the pair 6144 or 4096: its end, one tile more, two and several
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("N,K", [(50, 12288), (50, 12289), (50, 12416), (50, 28672), (4100, 8192), (4100, 8200), (4100, 8320),
                                 (4100, 16511)])
def test_columns_in_several_chunks(N, K, M, group):
    form_case(M, N, K, group, M == 1, "bf16" if K % 2 else "f16", False)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("N,K", [(50, 6144), (50, 6145), (50, 6272), (50, 13824), (4100, 4096), (4100, 4104), (4100, 5120),
                                 (4100, 8319)])
def test_columns_of_a_pair_in_several_chunks(N, K, M, group):
    form_case(M, N, K, group, M == 1, "bf16" if K % 2 else "f16", True)


@pytest.mark.parametrize("pair", [False, True])
def test_rows_across_batch_sizes(pair):
    """Above 4096 weight rows the sums of up to 4 rows are split over 8 waves, those of more over 16: equal within both
    sums' bounds. The same call gives the same bits."""
    N, K, group = 4100, 5000, 64
    gen = torch.Generator(device=dev())
    gen.manual_seed(3)
    ws = [device_weight(gen, N, K, group, True) for _ in range(2)]
    x = rows(np.random.default_rng(1060).standard_normal((16, K)), "f16")
    call = lambda t: (rb.q4_glu(ws[0][1], ws[1][1], t, N, group=group, act="none", y_dtype=torch.float32) if pair else  # noqa: E731
                      rb.q4_gemv(*ws[0][1], t, N, group=group, y_dtype=torch.float32))
    at = some_rows(N)
    i, xs = torch.from_numpy(at).to(dev()), n64(x)
    host = [of_rows(*w, at) for w in ws]
    V, L = ([f(h) for h in host] for f in (lambda h: xs @ BO.q4_values(*h, group).T, lambda h: product_bound(xs, h[1], h[2], group, K)))
    lim = 2 * (L[0] * (np.abs(V[1]) + L[1]) + np.abs(V[0]) * L[1] + 2 * U * np.abs(V[0] * V[1])) if pair else 2 * L[0]
    full = call(x)
    for m in (1, 2, 4, 7):
        got, again = call(x[:m]), call(x[:m])
        torch.cuda.synchronize()
        assert torch.equal(got, again)
        assert np.all(np.abs(n64(got[:, i]) - n64(full[:m, i])) <= lim[:m])


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("M", [1, 3, 16])
def test_weight_rows_past_one_part(M, pair):
    """More than 2^20 blocks of 16 weight rows: launched in parts. Every output is written, sampled ones are right."""
    N, K, group = (1 << 24) + 137, 96, 32
    gen = torch.Generator(device=dev())
    gen.manual_seed(M)
    ws = []
    for _ in range(1 + pair):
        codes = torch.randint(-(1 << 31), (1 << 31) - 1, (-(-N // 16), 1, 64, 4), dtype=torch.int32, generator=gen, device=dev())
        codes[..., 3] = 0  # columns 96 to 127
        codes.view(-1, 4, 16, 4)[-1, :, N % 16:] = 0  # rows past the last
        ws.append((codes, (torch.rand((3, N), generator=gen, device=dev()) * 0.01).half(), torch.randn((3, N), generator=gen, device=dev()).mul_(0.05).half()))
    x = rows(np.random.default_rng(1070).standard_normal((M, K)), "f16")
    y = torch.full((M, N), float("nan"), dtype=torch.float32, device=dev())
    if pair:
        rb.q4_glu(*ws, x, N, group=group, act="none", y=y)
    else:
        rb.q4_gemv(*ws[0], x, N, group=group, y=y)
    assert not torch.isnan(y).any()
    at = np.r_[0:20, (1 << 24) - 20:(1 << 24) + 20, N - 20:N]
    i, c, xs = torch.from_numpy(at).to(dev()), np.arange(K), n64(x)
    V, L = [], []
    for codes, s, z in ws:
        w = codes[i // 16, 0].cpu().numpy().view(np.uint32)  # [rows][lane][word]
        q = w[np.arange(at.size)[:, None], 16 * (c % 32 // 8)[None] + (at % 16)[:, None], (c // 32)[None]]
        q = q >> (16 * (c % 2) + 4 * (c % 8 // 2)).astype(np.uint32) & 15
        h = q.astype(np.int64), s[:, i].cpu().numpy(), z[:, i].cpu().numpy()
        V.append(xs @ BO.q4_values(*h, group).T)
        L.append(product_bound(xs, h[1], h[2], group, K))
    if pair:
        near(y[:, i], V[0] * V[1], L[0] * (np.abs(V[1]) + L[1]) + np.abs(V[0]) * L[1] + 2 * U * np.abs(V[0] * V[1]), "y")
    else:
        near(y[:, i], V[0], L[0], "y")
    del ws, y
    torch.cuda.empty_cache()
