"""GPU parity of the multi-tensor AdamW step (rb_adamw_plan / rb_adamw_step) against the oracle.

Comparison rules, u = 2^-24 the fp32 unit roundoff:
* m and v (32-bit states) are two products and a sum (a third product for g^2, one more for
  grad_scale): |error| <= 4 u (b1 |m| + (1 - b1) |g'|), 6 u (b2 v + (1 - b2) g'^2);
* p: the decayed term is rounded 3 times (the factor, the product, the difference) and the step's
  quotient has the relative errors of m above, of sqrt(v) (3.5 u), of the root, the product with
  the correction, the sum, the reciprocal (2 u), three products and the constants: 20 u of
  lr_t * (b1 |m| + (1 - b1) |g'|) / (1 - b1^t) / denominator covers them; fp16 and bf16 parameters
  add half a unit of their own;
* 8-bit states: scales are exact (the inputs keep the group maxima away from powers of two); each
  code is the oracle's stochastic rounding with the same random bits, unless the fp64 quotient lies
  within its fp32 error of the threshold, where the code on the other side of it is allowed too.
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
UNIT = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


def draw(seed, n, p_dt="f32", g_dt="f32", offset=0):
    """Parameter, gradient and fp32 states of n elements, each `offset` elements into its buffer."""
    r = np.random.default_rng([900, seed])
    def put(a, dt):
        buf = torch.zeros(n + offset, dtype=DT[dt], device=dev())
        buf[offset:] = torch.from_numpy(a.astype(np.float32)).to(DT[dt]).to(dev())
        return buf[offset:]
    g = r.standard_normal(n) * np.exp(r.standard_normal(n) - 6)
    g[r.random(n) < 0.05] = 0.0
    return (put(r.standard_normal(n) * 0.02, p_dt), put(g, g_dt), put(r.standard_normal(n) * 1e-3, "f32"),
            put(r.uniform(0.5, 2.0, n) ** 2 * 1e-6, "f32"))


def check32(before, after, step, wd=0.0, lr_mult=1.0, gs=1.0, p_dt="f32"):
    (p0, g, m0, v0), (p, m, v) = [np64(t) for t in before], [np64(t) for t in after]
    b1, b2, lr, eps = HYPER["beta1"], HYPER["beta2"], HYPER["lr"] * lr_mult, HYPER["eps"]
    po, mo, vo = BO.adamw(p0, g, m0, v0, step, lr, b1, b2, eps, wd, gs)
    mt = b1 * np.abs(m0) + (1 - b1) * np.abs(g * gs)
    assert np.all(np.abs(m - mo) <= 4 * U * mt + 2.0 ** -148)
    assert np.all(np.abs(v - vo) <= 6 * U * vo + 2.0 ** -148)
    den = np.sqrt(vo / (1 - b2 ** step)) + eps
    lim = 3 * U * np.abs(p0) + 20 * U * lr * mt / (1 - b1 ** step) / den + U * np.abs(po)
    lim += (UNIT[p_dt] * np.abs(po) if p_dt != "f32" else 0.0) + TINY[p_dt]
    assert np.all(np.abs(p - po) <= lim), np.max(np.abs(p - po) / lim)


@pytest.mark.parametrize("p_dt,g_dt", [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f32"),
                                       ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_step_types_and_odd_sizes(p_dt, g_dt):
    """Tensors of 1 to over two chunks in one plan, an empty one among them, some not aligned."""
    sizes = [1, 3, 0, 255, 256, 257, 1000, 4095, 4096, 4097, 9001]
    parts = [draw(i, n, p_dt, g_dt, offset=(0, 1, 2, 3)[i % 4]) for i, n in enumerate(sizes)]
    before = [[t.clone() for t in x] for x in parts]
    wd = [0.1 * (i % 2) for i in range(len(sizes))]
    lm = [1.0 if i % 3 else 0.25 for i in range(len(sizes))]
    plan = rb.adamw_plan([x[0] for x in parts], [x[1] for x in parts], m=[x[2] for x in parts], v=[x[3] for x in parts],
                         weight_decay=wd, lr_mult=lm)
    rb.adamw_step(plan, 7, **HYPER)
    torch.cuda.synchronize()
    for x, b, w, l in zip(parts, before, wd, lm):
        if x[0].numel():
            check32(b, (x[0], x[2], x[3]), 7, w, l, p_dt=p_dt)
            assert torch.equal(x[1], b[1]), "the gradient changed"


def test_writes_stay_inside_the_tensors():
    n = 4099
    bufs = [torch.full((n + 16,), 7.0, device=dev()) for _ in range(4)]
    views = [b[5:5 + n] for b in bufs]
    for v, x in zip(views, draw(50, n)):
        v.copy_(x)
    plan = rb.adamw_plan([views[0]], [views[1]], m=[views[2]], v=[views[3]])
    rb.adamw_step(plan, 1, **HYPER)
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.all(b[:5] == 7.0) and torch.all(b[5 + n:] == 7.0)


def test_grad_scale_and_skip():
    parts = draw(60, 5000)
    before = [t.clone() for t in parts]
    plan = rb.adamw_plan([parts[0]], [parts[1]], m=[parts[2]], v=[parts[3]])
    gs, skip = torch.tensor([0.3], device=dev()), torch.tensor([1], dtype=torch.int32, device=dev())
    rb.adamw_step(plan, 3, grad_scale=gs, skip=skip, **HYPER)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(parts, before)), "a skipped step changed something"
    skip.zero_()
    rb.adamw_step(plan, 3, grad_scale=gs, skip=skip, **HYPER)
    torch.cuda.synchronize()
    check32(before, (parts[0], parts[2], parts[3]), 3, gs=float(np64(gs)[0]))


def test_many_steps_from_zero_follow_the_oracle():
    """20 steps of fresh states on a fixed gradient sequence; the errors of single steps add."""
    n, steps = 3000, 20
    p, g, _, _ = draw(70, n)
    plan = rb.adamw_plan([p], [g], weight_decay=0.1)
    po, mo, vo = np64(p), np.zeros(n), np.zeros(n)
    for t in range(1, steps + 1):
        g.copy_(draw(70 + t, n)[1])
        po, mo, vo = BO.adamw(po, np64(g), mo, vo, t, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], 0.1)
        rb.adamw_step(plan, t, **HYPER)
    torch.cuda.synchronize()
    # per step: 4 u of p and 40 u of a step no longer than lr * 10 (|m| <= 10 sqrt(v) in these sequences)
    lim = steps * (4 * U * (np.abs(po) + 0.1) + 40 * U * HYPER["lr"] * 10)
    assert np.all(np.abs(np64(plan.params[0]) - po) <= lim)


def test_non_finite_gradients_stay_in_their_element():
    parts = draw(80, 1000)
    parts[1][10], parts[1][700] = float("nan"), float("inf")
    before = [t.clone() for t in parts]
    plan = rb.adamw_plan([parts[0]], [parts[1]], m=[parts[2]], v=[parts[3]])
    rb.adamw_step(plan, 2, **HYPER)
    torch.cuda.synchronize()
    for t in (parts[0], parts[2], parts[3]):
        bad = ~torch.isfinite(t)
        assert bad.nonzero().flatten().tolist() == [10, 700]
    keep = torch.ones(1000, dtype=torch.bool, device=dev())
    keep[[10, 700]] = False
    check32([t[keep] for t in before], [t[keep] for t in (parts[0], parts[2], parts[3])], 2)


# ---------------------------------------------------------------------------------------------
# 8-bit states
# ---------------------------------------------------------------------------------------------
def draw8(seed, n, offset=0):
    """8-bit states of n elements, some groups all zero, with their scales."""
    r = np.random.default_rng([901, seed])
    rows = (n + 255) // 256
    def codes(signed):
        c = r.integers(0, 0x79, n).astype(np.uint8)
        if signed:
            c |= (r.integers(0, 2, n) << 7).astype(np.uint8)
        if rows > 2:
            c[256:512] = 0
        buf = torch.zeros(n + offset, dtype=torch.uint8, device=dev())
        buf[offset:] = torch.from_numpy(c).to(dev())
        return buf.view(torch.float8_e4m3fn)[offset:]
    def scales():
        return torch.from_numpy(np.ldexp(1.0, r.integers(-12, -6, rows)).astype(np.float32)).to(dev())
    return codes(True), codes(False), scales(), scales()


def check_codes(x, err, codes, scales, rnd16, low):
    """x: the fp64 values, err: bounds of their fp32 errors; rnd16: the random halves."""
    so = BO.adamw_scales(x)
    assert np.array_equal(scales, so), "scales differ"
    a, grid = BO.adamw_grid(x, so)
    d = err / np.repeat(so, 256)[:x.size] * 256.0 / grid + 2.0 ** -19  # and the subnormal cut of the quotient
    t = a / grid + (rnd16 + 0.5) / 65536.0
    lo, hi = np.floor(t - d) * grid, np.floor(t + d) * grid
    if low:
        lo, hi = (np.where(x != 0, np.maximum(b, 2.0 ** -9), b) for b in (lo, hi))
    got = np.abs(BO.E4M3[codes])
    bad = (got < lo) | (got > hi)
    assert not bad.any(), (bad.sum(), np.flatnonzero(bad)[:3], got[bad][:3], lo[bad][:3], hi[bad][:3])
    assert np.all((np.signbit(x) == (codes >= 128)) | (x == 0))
    return float(np.mean(lo != hi))


@pytest.mark.parametrize("offset", [0, 1])
def test_8bit_step_follows_the_definition(offset):
    sizes = [1, 255, 4096, 700, 5001]
    st = [draw8(i, n, offset) for i, n in enumerate(sizes)]
    pg = [draw(20 + i, n)[:2] for i, n in enumerate(sizes)]
    before = [[t.clone() for t in (*a, *b)] for a, b in zip(pg, st)]
    plan = rb.adamw_plan([x[0] for x in pg], [x[1] for x in pg], state_bits=8, m=[x[0] for x in st],
                         v=[x[1] for x in st], m_scale=[x[2] for x in st], v_scale=[x[3] for x in st], weight_decay=0.1)
    step, seed = 5, 1234567
    rb.adamw_step(plan, step, seed=seed, **HYPER)
    torch.cuda.synchronize()
    chunk, b1, b2 = 0, HYPER["beta1"], HYPER["beta2"]
    for n, (p, g), (mc, vc, ms, vs), b in zip(sizes, pg, st, before):
        m0 = BO.adamw_decode(b[2].view(torch.uint8).cpu().numpy(), np64(b[4]))
        r0 = BO.adamw_decode(b[3].view(torch.uint8).cpu().numpy(), np64(b[5]))
        p0, g0 = np64(b[0]), np64(b[1])
        po, mo, vo = BO.adamw(p0, g0, m0, r0 * r0, step, HYPER["lr"], b1, b2, HYPER["eps"], 0.1)
        mt = b1 * np.abs(m0) + (1 - b1) * np.abs(g0)
        h = BO.adamw_random(chunk * 4096 + np.arange(n), step, seed)
        near = [check_codes(mo, 4 * U * mt, mc.view(torch.uint8).cpu().numpy(), np64(ms), h & 0xFFFF, False),
                check_codes(np.sqrt(vo), 5 * U * np.sqrt(vo), vc.view(torch.uint8).cpu().numpy(), np64(vs), h >> 16, True)]
        assert max(near) < 0.01 or n < 1000, "the random bits decide nearly every code"
        den = np.sqrt(vo / (1 - b2 ** step)) + HYPER["eps"]
        lim = 4 * U * np.abs(p0) + 20 * U * HYPER["lr"] * mt / (1 - b1 ** step) / den + U * np.abs(po)
        assert np.all(np.abs(np64(p) - po) <= lim)
        chunk += (n + 4095) // 4096


def test_8bit_step_past_32_bits():
    """One tensor of over 2^32 elements: offsets, scales and the random numbers' positions on both sides of 2^32."""
    n, step, seed = (1 << 32) + 3 * 4096 + 77, 3, 99
    torch.manual_seed(106)
    p, g = torch.empty(n, dtype=torch.bfloat16, device=dev()).normal_(), torch.empty(n, dtype=torch.bfloat16, device=dev()).normal_()
    m, v = (torch.randint(0, 0x79, (n,), dtype=torch.uint8, device=dev()) for _ in range(2))
    ms, vs = (torch.full(((n + 255) // 256,), 0.5, device=dev()) for _ in range(2))
    parts = [slice(0, 512), slice((1 << 32) - 512, (1 << 32) + 512), slice(n - 77 - 256, n)]
    group = [slice(s.start // 256, (s.stop + 255) // 256) for s in parts]
    before = [[np64(p[s]), np64(g[s]), m[s].cpu().numpy(), v[s].cpu().numpy()] for s in parts]
    plan = rb.adamw_plan([p], [g], state_bits=8, m=[m.view(torch.float8_e4m3fn)], v=[v.view(torch.float8_e4m3fn)],
                         m_scale=[ms], v_scale=[vs])
    rb.adamw_step(plan, step, seed=seed, **HYPER)
    torch.cuda.synchronize()
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    for s, q, (p0, g0, mc, vc) in zip(parts, group, before):
        half = np.full(q.stop - q.start, 0.5)
        m0, r0 = BO.adamw_decode(mc, half), BO.adamw_decode(vc, half)
        po, mo, vo = BO.adamw(p0, g0, m0, r0 * r0, step, HYPER["lr"], b1, b2, HYPER["eps"])
        mt = b1 * np.abs(m0) + (1 - b1) * np.abs(g0)
        h = BO.adamw_random(np.arange(s.start, s.stop), step, seed)
        # bf16 gradients meet the states' few values: sums that cancel to within their own error may have either sign
        codes = m[s].cpu().numpy()
        mo = np.where(np.abs(mo) <= 4 * U * mt, np.copysign(mo, BO.E4M3[codes]), mo)
        check_codes(mo, 4 * U * mt, codes, np64(ms[q]), h & 0xFFFF, False)
        check_codes(np.sqrt(vo), 5 * U * np.sqrt(vo), v[s].cpu().numpy(), np64(vs[q]), h >> 16, True)
        den = np.sqrt(vo / (1 - b2 ** step)) + HYPER["eps"]
        lim = 3 * U * np.abs(p0) + 20 * U * HYPER["lr"] * mt / (1 - b1 ** step) / den + (U + UNIT["bf16"]) * np.abs(po)
        assert np.all(np.abs(np64(p[s]) - po) <= lim + TINY["bf16"])
    del p, g, m, v, plan
    torch.cuda.empty_cache()


def test_8bit_unchanged_state_is_stored_unchanged():
    """1 - 2^-53 rounds to 1: with no gradient the states stay, and their values must be stored again
    exactly. A group whose largest magnitude equals its scale (code 0x78) takes the next power of two,
    where the values of odd subnormal codes no longer fit; all others must be the same."""
    n = 2000
    m, v, ms, vs = draw8(30, n)
    for c in (m, v):   # a large code in every group, so the scale is its own or the next
        c.view(torch.uint8)[::256] = 0x77
    p, g = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    value = lambda c, s: BO.adamw_decode(c.view(torch.uint8).cpu().numpy(), np64(s))  # noqa: E731
    before = [value(m, ms), value(v, vs)]
    plan = rb.adamw_plan([p], [g], state_bits=8, m=[m], v=[v], m_scale=[ms], v_scale=[vs])
    rb.adamw_step(plan, 1, 1e-3, beta1=1 - 2.0 ** -53, beta2=1 - 2.0 ** -53)
    torch.cuda.synchronize()
    for c, s, x in ((m, ms, before[0]), (v, vs, before[1])):
        scales = BO.adamw_scales(x)
        assert np.array_equal(np64(s), scales)
        a, grid = BO.adamw_grid(x, scales)
        fits = a / grid == np.floor(a / grid)
        assert fits.mean() > 0.9
        assert np.array_equal(value(c, s)[fits], x[fits])


def test_8bit_rounding_is_unbiased_and_decays():
    """256 elements at the group's maximum and one tensor of equal small values under decay alone
    (no gradient): sqrt(v) follows beta2^(t/2) although each step is far below half a code. The mean of
    n = 65536 elements after 60 steps: one rounding has a standard deviation of at most half a code,
    1/16 of the value; 60 of them, averaged over n, stay within 6 deviations of the exact decay."""
    n, steps = 65536, 60
    p, g = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    v = torch.full((n,), 64.0, device=dev()).to(torch.float8_e4m3fn)
    v[::256] = 240.0
    m = torch.zeros(n, device=dev()).to(torch.float8_e4m3fn)
    one = torch.ones(n // 256, device=dev())
    plan = rb.adamw_plan([p], [g], state_bits=8, m=[m], v=[v], m_scale=[one.clone()], v_scale=[one.clone()])
    for t in range(1, steps + 1):
        rb.adamw_step(plan, t, 1e-3, beta2=0.999, seed=9)
    torch.cuda.synchronize()
    got = BO.adamw_decode(v.view(torch.uint8).cpu().numpy(), np64(plan.v_scale[0])).reshape(-1, 256)[:, 1:]
    want = 0.25 * 0.999 ** (steps / 2)
    sd = want / 16 * np.sqrt(steps) / np.sqrt(got.size)
    assert abs(got.mean() - want) <= 6 * sd, (got.mean(), want, sd)


def test_8bit_non_finite_and_tiny():
    n = 512
    p, g = draw(90, n)[:2]
    g[3], g[300] = float("nan"), float("-inf")
    before = p.clone()
    plan = rb.adamw_plan([p], [g], state_bits=8)
    rb.adamw_step(plan, 1, seed=2, **HYPER)
    torch.cuda.synchronize()
    for c in (plan.m[0], plan.v[0], p):
        assert (~torch.isfinite(c.float())).nonzero().flatten().tolist() == [3, 300]
    assert torch.isfinite(plan.m_scale[0]).all() and torch.isfinite(plan.v_scale[0]).all()
    # a value far below its group's largest keeps a nonzero root, so the next step stays bounded
    g.zero_()
    g[0], g[1] = 1.0, 1e-7
    p.copy_(before)
    plan = rb.adamw_plan([p], [g], state_bits=8)
    for t in (1, 2, 3):
        rb.adamw_step(plan, t, seed=2, **HYPER)
    torch.cuda.synchronize()
    assert plan.v[0][1].float() > 0
    assert torch.all(torch.abs(p - before) <= 3 * HYPER["lr"] * 4)


def test_8bit_is_deterministic_and_seeded():
    outs = []
    for seed in (5, 5, 6):
        p, g = draw(100, 9000)[:2]
        plan = rb.adamw_plan([p], [g], state_bits=8)
        for t in (1, 2):
            rb.adamw_step(plan, t, seed=seed, **HYPER)
        torch.cuda.synchronize()
        outs.append([t.clone().view(torch.uint8) for t in (plan.m[0], plan.v[0])] + [p.clone()])
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    assert not torch.equal(outs[0][0], outs[2][0])


def test_runs_on_the_current_stream_and_in_a_graph():
    parts = draw(110, 20000)
    before = [t.clone() for t in parts]
    plan = rb.adamw_plan([parts[0]], [parts[1]], m=[parts[2]], v=[parts[3]])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rb.adamw_step(plan, 4, **HYPER)
    s.synchronize()
    check32(before, (parts[0], parts[2], parts[3]), 4)
    want = [t.clone() for t in parts]
    graph = torch.cuda.CUDAGraph()
    for t, b in zip(parts, before):
        t.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rb.adamw_step(plan, 4, **HYPER)
    for _ in range(3):
        for t, b in zip(parts, before):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(parts, want))


def test_plan_refusals():
    p, g, m, v = draw(120, 100)
    with pytest.raises(ValueError):
        rb.adamw_plan([], [])
    with pytest.raises(ValueError):
        rb.adamw_plan([p], [g[:50]])
    with pytest.raises(ValueError):
        rb.adamw_plan([p], [g, g])
    with pytest.raises(ValueError):
        rb.adamw_plan([p], [g], state_bits=16)
    with pytest.raises(ValueError):
        rb.adamw_plan([p], [g], state_bits=8, m=[m], v=[v])          # fp32 states
    with pytest.raises(ValueError):
        rb.adamw_plan([p[::2]], [g[::2]])                            # not contiguous
    with pytest.raises(ValueError):
        rb.adamw_plan([p.cpu()], [g.cpu()])
    with pytest.raises(rb.RbError):
        rb.adamw_plan([p.half()], [g.bfloat16()])
    plan = rb.adamw_plan([p], [g], m=[m], v=[v])
    with pytest.raises(rb.RbError):
        rb.adamw_step(plan, 0, 1e-3)
    with pytest.raises(rb.RbError):
        rb.adamw_step(plan, 1, 1e-3, beta1=1.0)
    with pytest.raises(TypeError):
        rb.adamw_step(plan, 1, 1e-3, skip=torch.zeros(1, device=dev()))
