"""The operators of a gated feed-forward block, from its training to its serving, and how they are measured.

Each in its plain form (torch, 32 bits) and as a call of the library:

* glu:      G = X Wg^T + bg, U = X Wu^T + bu, H = act(G) U;
* glu_bwd:  its backward: dG = dH U act'(G), dU = dH act(G) (rounded to the activations' type, as the next
            products take them), the biases' gradients, and dX = dG Wg + dU Wu;
* muon:     one optimizer step of a matrix by momentum and five Newton-Schulz products;
* q4:       y = W x with 4-bit weights and group scales, or the gated pair H = act(Wg x) (Wu x);
* q4_pack:  weights to 4 bits and back.

``own`` selects the form. Inputs are seeded.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315  # the odd polynomial of one Newton-Schulz product
NS_STEPS, NS_EPS = 5, 1e-7
LR, MU, DECAY = 3e-4, 0.95, 0.1
TILE_N, TILE_K = 16, 128  # weight rows and columns of one tile of packed 4-bit codes


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _glu(M, N, K, dt, act, bias, h_dt, save, pad=0):
    return dict(op="glu", M=M, N=N, K=K, dt=dt, act=act, bias=bias, h_dt=h_dt, save=save, pad=pad)


def _glu_bwd(M, N, K, dt, act, bias, dh_dt, pad=0):
    return dict(op="glu_bwd", M=M, N=N, K=K, dt=dt, act=act, bias=bias, dh_dt=dh_dt, pad=pad)


def _muon(N, K, nesterov, scale):
    return dict(op="muon", N=N, K=K, nesterov=nesterov, scale=scale)


def _q4(M, N, K, group, offset, dt, y_dt, pair, act="none"):
    return dict(op="q4", M=M, N=N, K=K, group=group, offset=offset, dt=dt, y_dt=y_dt, pair=pair, act=act)


def _q4_pack(N, K, group, offset, w_dt, dt):
    return dict(op="q4_pack", N=N, K=K, group=group, offset=offset, w_dt=w_dt, dt=dt)


def listed():
    return [
        # one token through the gate and up projections: a decode step on effective weights, latency and bandwidth
        dict(_glu(1, 11008, 4096, "f16", "silu", False, "f16", False), name="glu 1 token"),
        # a short batch on an odd block whose rows are not 16-byte aligned, pre-activations kept
        dict(_glu(61, 1411, 1027, "bf16", "gelu_tanh", True, "f32", True), name="glu ragged 61x1411x1027"),
        # a training batch, pre-activations kept for the backward
        dict(_glu(2048, 11008, 4096, "bf16", "silu", False, "bf16", True), name="glu 2048 tokens"),
        # the backward of the odd block and of the training batch
        dict(_glu_bwd(61, 1411, 1027, "bf16", "gelu_tanh", True, "f32"), name="glu backward ragged"),
        dict(_glu_bwd(2048, 11008, 4096, "bf16", "silu", False, "bf16"), name="glu backward 2048 tokens"),
        # a small layer's matrix: nine dependent products of little work, latency
        dict(_muon(256, 512, True, False), name="muon 256x512"),
        # the up and the down projection's shared weight; the tall one is orthogonalised as its transpose
        dict(_muon(11008, 4096, True, True), name="muon 11008x4096"),
        # one token through a down projection in 4 bits
        dict(_q4(1, 4096, 11008, 128, False, "f16", "f16", False), name="q4 1 token 4096x11008"),
        # a decode batch on an odd layer, small groups with offsets
        dict(_q4(16, 4095, 11007, 32, True, "bf16", "bf16", False), name="q4 16 tokens 4095x11007"),
        # one token through the gated pair in 4 bits
        dict(_q4(1, 11008, 4096, 128, False, "bf16", "bf16", True, "silu"), name="q4 gated pair 1 token"),
        # quantising a trained projection, and the effective weight a long prompt's product takes
        dict(_q4_pack(4096, 11008, 128, True, "f32", "bf16"), name="q4 pack 4096x11008"),
        dict(_q4_pack(1027, 1411, 32, False, "bf16", "f16"), name="q4 pack odd 1027x1411"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm; half of them multiples of 160, the others as they fall."""
    n = _log(rng, lo, hi)
    return n // 160 * 160 if n >= 160 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_bwd", "glu_bwd", "muon", "muon", "q4", "q4", "q4_pack"])
    dt = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op in ("glu", "glu_bwd"):
        while True:
            M, N, K = _log(rng, 1, 4096), _size(rng, 200, 11008), _size(rng, 200, 11008)
            if M * N * K <= 2048 * 4096 * 11008:
                break
        pad = rng.choice([0, 0, 8, 3])
        if op == "glu":
            return _glu(M, N, K, dt, act, rng.random() < 0.3, rng.choice([dt, dt, "f32"]), rng.random() < 0.5, pad)
        return _glu_bwd(M, N, K, dt, act, rng.random() < 0.3, rng.choice([dt, "f32"]), pad)
    if op == "muon":
        while True:
            N, K = _size(rng, 64, 11008), _size(rng, 64, 11008)
            if min(N, K) ** 2 * (min(N, K) + 3 * max(N, K)) <= 4096 ** 2 * (4096 + 3 * 11008):
                break
        return _muon(N, K, rng.random() < 0.7, rng.random() < 0.5)
    while True:
        N, K = _size(rng, 200, 11008), _size(rng, 200, 11008)
        if N * K <= 4096 * 11008:
            break
    group, offset = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "q4":
        pair = rng.random() < 0.4
        return _q4(_log(rng, 1, 16), N, K, group, offset, dt, rng.choice([dt, dt, "f32"]), pair, act if pair else "none")
    return _q4_pack(N, K, group, offset, rng.choice(["f32", "f32", dt]), dt)


def work(c):
    """Each input read once, each output written once; a symmetric product is half of one."""
    N, K = c["N"], c["K"]
    if c["op"] == "glu":
        M, e = c["M"], SIZE[c["dt"]]
        b = (M * K + 2 * N * K) * e + M * N * (SIZE[c["h_dt"]] + 2 * e * c["save"]) + 8 * N * c["bias"]
        return {"bytes": b, "flops": 4 * M * N * K}
    if c["op"] == "glu_bwd":
        M, e = c["M"], SIZE[c["dt"]]
        b = M * N * (SIZE[c["dh_dt"]] + 4 * e) + (M * K + 2 * N * K) * e + 8 * N * c["bias"]
        return {"bytes": b, "flops": 4 * M * N * K + 15 * M * N}
    if c["op"] == "muon":
        n, m = min(N, K), max(N, K)
        return {"bytes": 20 * N * K, "flops": NS_STEPS * n * n * (n + 3 * m)}
    groups = (K + c["group"] - 1) // c["group"]
    held = N * K // 2 + 2 * N * groups * (1 + c["offset"])
    if c["op"] == "q4":
        two = 1 + c["pair"]
        return {"bytes": two * held + c["M"] * (K * SIZE[c["dt"]] + N * SIZE[c["y_dt"]]), "flops": 2 * two * c["M"] * N * K}
    return {"bytes": N * K * (SIZE[c["w_dt"]] + SIZE[c["dt"]]) + 2 * held, "flops": 8 * N * K}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dt, std=1.0, pad=0):
    """N(0, std^2) rows; with a pad, a view of rows that lie pad elements further apart."""
    t = torch.randn((*shape[:-1], shape[-1] + pad), generator=g, device="cuda").mul_(std).to(dt)
    return t[..., :shape[-1]] if pad else t


def _vector(g, n, lo, hi):
    return torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo


def _effective_weight(g, N, K, dt, pad):
    """Two residual paths: row scales near 0.016 and half of that, column scales near 1, random signs."""
    w = None
    for i in range(2):
        sign = (torch.rand((N, K + pad), generator=g, device="cuda") < 0.5).float().mul_(2).sub_(1)
        path = sign.mul_((_vector(g, N, 0.5, 1.5) * (0.016 * 0.5 ** i))[:, None]).mul_(_vector(g, K + pad, 0.5, 1.5))
        w = path if w is None else w.add_(path)
    w = w.to(dt)
    return w[:, :K] if pad else w


def _gradient(g, N, K, std):
    """A weight's gradient: most of it of a rank far below full, rows of different sizes."""
    r = max(1, min(N, K) // 16)
    low = torch.randn((N, r), generator=g, device="cuda") @ torch.randn((r, K), generator=g, device="cuda")
    noise = torch.randn((N, K), generator=g, device="cuda").mul_(0.3)
    return low.mul_(r ** -0.5).add_(noise).mul_(_vector(g, N, 0.3, 1.7)[:, None] * std)


def _codes(q):
    """Codes [N][K] to the packed layout [N / 16][K / 128][64][4] of 32-bit words: lane 16 j + r of a tile holds row r,
    its word i columns 32 i + 8 j .. + 7, column c of those in the four bits from 16 (c % 2) + 4 (c / 2) on."""
    N, K = q.shape
    tn, tk = -(-N // TILE_N), -(-K // TILE_K)
    full = torch.zeros((tn * TILE_N, tk * TILE_K), dtype=torch.int64, device=q.device)
    full[:N, :K] = q
    t = full.view(tn, TILE_N, tk, 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 6, 5)  # tile, tile, j, r, i, c % 2, c / 2
    w = (t << (4 * torch.arange(8, device=q.device).view(2, 4))).sum((-1, -2))
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).reshape(tn, tk, 64, 4).contiguous()


def _uncode(words, N, K):
    """The codes [N][K] (int32) of the packed layout."""
    tn, tk = words.shape[:2]
    shift = 4 * torch.arange(8, dtype=torch.int32, device=words.device).view(2, 4)
    t = (words.view(tn, tk, 4, TILE_N, 4, 1, 1) >> shift) & 15
    return t.permute(0, 3, 1, 4, 2, 6, 5).reshape(tn * TILE_N, tk * TILE_K)[:N, :K]


def _groups(w, group):
    """Rows in whole groups, the last filled up with its row's last value: [N][groups][group]."""
    N, K = w.shape
    n = -(-K // group)
    return torch.cat([w, w[:, -1:].expand(N, n * group - K)], 1).view(N, n, group)


def _quantise(W, group, offset):
    """(codes [N][K], s [groups][N], z [groups][N] or None), scales in fp16, arithmetic in 32 bits."""
    N, K = W.shape
    w = _groups(W.float(), group)
    if offset:
        lo, hi = w.amin(2), w.amax(2)
        z = lo.half()
        s = ((hi - lo) / 15.0).half()
        d, first, last = w - z.float()[..., None], 0.0, 15.0
    else:
        z, s = None, (w.abs().amax(2) / 7.0).half()
        d, first, last = w, -8.0, 7.0
    q = torch.where(s[..., None] > 0, torch.round(d / s.float()[..., None]), 0.0).clamp(first, last) - first
    q = q.reshape(N, -1)[:, :K]
    return q.to(torch.int32), s.t().contiguous(), None if z is None else z.t().contiguous()


def _values(q, s, z, group):
    """The weights (32 bits) that codes stand for."""
    N, K = q.shape
    each = lambda t: t.float().t().repeat_interleave(group, 1)[:, :K]  # noqa: E731
    return each(s) * (q - 8) if z is None else each(s) * q + each(z)


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    N, K = c["N"], c["K"]
    if c["op"] in ("glu", "glu_bwd"):
        M, dt = c["M"], DT[c["dt"]]
        s["Wg"], s["Wu"] = (_effective_weight(g, N, K, dt, c["pad"]) for _ in range(2))
        if c["op"] == "glu":
            s["X"] = _normal(g, (M, K), dt, pad=c["pad"])
            s["bg"], s["bu"] = (_normal(g, (N,), torch.float32, 0.1) if c["bias"] else None for _ in range(2))
            s["H"] = torch.empty((M, N), dtype=DT[c["h_dt"]], device="cuda")
            s["G"], s["U"] = (torch.empty((M, N), dtype=dt, device="cuda") if c["save"] else None for _ in range(2))
        else:
            s["dH"] = _normal(g, (M, N), DT[c["dh_dt"]], 0.01)
            s["G"], s["U"] = (_normal(g, (M, N), dt, 1.2) for _ in range(2))
            s["dG"], s["dU"] = (torch.empty((M, N), dtype=dt, device="cuda") for _ in range(2))
            s["dX"] = torch.empty((M, K), dtype=dt, device="cuda")
    elif c["op"] == "muon":
        # a training run some steps in
        s["W"] = _normal(g, (N, K), torch.float32, 0.02)
        s["grad"], s["mom"] = _gradient(g, N, K, 1e-4), _gradient(g, N, K, 1e-3)
        s["grad_scale"] = _vector(g, 1, 0.5, 1.0) if c["scale"] else None
    elif c["op"] == "q4":
        dt = DT[c["dt"]]
        # activations with a few channels far above the others
        s["x"] = _normal(g, (c["M"], K), torch.float32).mul_(torch.where(_vector(g, K, 0, 1) < 0.01, 8.0, 1.0)).to(dt)
        s["W"] = []
        for _ in range(1 + c["pair"]):
            q, sc, z = _quantise(_normal(g, (N, K), torch.float32, 0.02), c["group"], c["offset"])
            s["W"].append((_codes(q), sc, z))
        s["y"] = torch.empty((c["M"], N), dtype=DT[c["y_dt"]], device="cuda")
    else:
        # trained weights: normal with heavier tails, rows and groups of different sizes
        w = torch.randn((N, K), generator=g, device="cuda")
        w.mul_(0.02).mul_(_vector(g, N, 0.5, 1.5)[:, None]).mul_(1 + 0.3 * torch.randn(K, generator=g, device="cuda").abs())
        s["W"] = w.to(DT[c["w_dt"]])
        s["What"] = torch.empty((N, K), dtype=DT[c["dt"]], device="cuda")
    return s


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import residual_binarized_weight_amd as rb
    c = s["c"]
    if c["op"] == "glu":
        H, G, U = rb.qat_glu(s["X"], s["Wg"], s["Wu"], act=c["act"], bias_g=s["bg"], bias_u=s["bu"], H=s["H"], G=s["G"],
                             U=s["U"])
        return {"H": H, "G": G, "U": U}
    if c["op"] == "glu_bwd":
        dG, dU, dbg, dbu = rb.qat_glu_backward(s["dH"], s["G"], s["U"], act=c["act"], bias=c["bias"], dG=s["dG"],
                                               dU=s["dU"])
        dX = rb.qat_glu_dx(dG, dU, s["Wg"], s["Wu"], dX=s["dX"])
        return {"dG": dG, "dU": dU, "dbg": dbg, "dbu": dbu, "dX": dX}
    if c["op"] == "muon":
        rb.muon_step(s["W"], s["grad"], s["mom"], LR, momentum=MU, nesterov=c["nesterov"], weight_decay=DECAY,
                     grad_scale=s["grad_scale"], steps=NS_STEPS, eps=NS_EPS)
        return {"W": s["W"], "mom": s["mom"]}
    if c["op"] == "q4":
        if c["pair"]:
            return rb.q4_glu(s["W"][0], s["W"][1], s["x"], c["N"], group=c["group"], act=c["act"], y=s["y"])
        return rb.q4_gemv(*s["W"][0], s["x"], c["N"], group=c["group"], y=s["y"])
    codes, sc, z = rb.q4_pack(s["W"], group=c["group"], offset=c["offset"])
    return {"What": rb.q4_dequant(codes, sc, z, c["N"], c["K"], group=c["group"], What=s["What"]), "s": sc, "z": z}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0 * z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _run_plain(s):
    c = s["c"]
    if c["op"] == "glu":
        x = s["X"].float()
        g, u = x @ s["Wg"].float().t(), x @ s["Wu"].float().t()
        if c["bias"]:
            g, u = g + s["bg"], u + s["bu"]
        kept = DT[c["dt"]] if c["save"] else None
        return {"H": (_act(g, c["act"]) * u).to(DT[c["h_dt"]]), "G": kept and g.to(kept), "U": kept and u.to(kept)}
    if c["op"] == "glu_bwd":
        dh, g, u = s["dH"].float(), s["G"].float(), s["U"].float()
        dg, du = dh * u * _act_slope(g, c["act"]), dh * _act(g, c["act"])
        dbg, dbu = (dg.sum(0), du.sum(0)) if c["bias"] else (None, None)
        dg, du = dg.to(DT[c["dt"]]), du.to(DT[c["dt"]])
        dx = dg.float() @ s["Wg"].float() + du.float() @ s["Wu"].float()
        return {"dG": dg, "dU": du, "dbg": dbg, "dbu": dbu, "dX": dx.to(DT[c["dt"]])}
    if c["op"] == "muon":
        return _plain_muon(s)
    if c["op"] == "q4":
        x = s["x"].float()
        y = [x @ _values(_uncode(codes, c["N"], c["K"]), sc, z, c["group"]).t() for codes, sc, z in s["W"]]
        return (_act(y[0], c["act"]) * y[1] if c["pair"] else y[0]).to(DT[c["y_dt"]])
    q, sc, z = _quantise(s["W"], c["group"], c["offset"])
    codes = _codes(q)  # what is kept of the weights
    return {"What": _values(_uncode(codes, c["N"], c["K"]), sc, z, c["group"]).to(DT[c["dt"]]), "s": sc, "z": z}


def _plain_muon(s):
    c = s["c"]
    g = s["grad"] if s["grad_scale"] is None else s["grad"] * s["grad_scale"]
    s["mom"] = MU * s["mom"] + g
    x = g + MU * s["mom"] if c["nesterov"] else s["mom"]
    tall = c["N"] > c["K"]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.t()
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    x = x.t() if tall else x
    s["W"] = s["W"] * (1 - LR * DECAY) - LR * 0.2 * math.sqrt(max(c["N"], c["K"])) * x
    return {"W": s["W"], "mom": s["mom"]}


# --------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------------------------
def exact(c, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if c["op"] == "glu":
        g, u = (torch.mm(f["X"], f[w].t().contiguous()) for w in ("Wg", "Wu"))
        if c["bias"]:
            g, u = g + f["bg"], u + f["bu"]
        h = _exact_act(g, c["act"])[0] * u
        return {"H": h, "G": g if c["save"] else None, "U": u if c["save"] else None}
    if c["op"] == "glu_bwd":
        value, slope = _exact_act(f["G"], c["act"])
        dg, du = slope * f["U"] * f["dH"], value * f["dH"]
        ones = torch.ones_like(dg[:, 0])
        sums = [torch.mv(d.t(), ones) if c["bias"] else None for d in (dg, du)]
        dx = torch.mm(torch.cat([dg, du], 1), torch.cat([f["Wg"], f["Wu"]], 0))
        return {"dG": dg, "dU": du, "dbg": sums[0], "dbu": sums[1], "dX": dx}
    if c["op"] == "muon":
        return _exact_muon(c, f)
    if c["op"] == "q4":
        y = [torch.mm(f["x"], _exact_weight(_exact_codes(w[0], c), w[1], w[2], c).t().contiguous()) for w in s["W"]]
        return _exact_act(y[0], c["act"])[0] * y[1] if c["pair"] else y[0]
    return _exact_pack(c, s)


def _exact_act(z, act):
    """(value, derivative)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(math.tau)
    if act == "silu":
        g = torch.sigmoid(z)
        return z * g, g + z * g * torch.sigmoid(-z)
    # (1 + tanh a) / 2 is the logistic function of 2a
    a = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    g = torch.sigmoid(a)
    return z * g, g + z * g * (1 - g) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)


def _exact_muon(c, f):
    """The polynomial's powers gathered on the smaller side: p(X) = (a + b A + c A^2) X, A the smaller Gram matrix."""
    g = f["grad"] * (1.0 if f["grad_scale"] is None else f["grad_scale"])
    mom = torch.add(g, f["mom"], alpha=MU)
    x = torch.add(g, mom, alpha=MU) if c["nesterov"] else mom
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    tall = c["N"] > c["K"]
    eye = torch.eye(min(c["N"], c["K"]), dtype=torch.float64, device="cuda")
    for _ in range(NS_STEPS):
        t = x.t().contiguous()
        a = torch.mm(t, x) if tall else torch.mm(x, t)
        p = torch.addmm(NS_A * eye, NS_C * a + NS_B * eye, a)
        x = torch.mm(x, p) if tall else torch.mm(p, x)
    return {"W": torch.lerp(f["W"], torch.zeros_like(x), LR * DECAY) - x * (LR * 0.2 * max(c["N"], c["K"]) ** 0.5), "mom": mom}


def _exact_codes(words, c):
    """Codes by dividing the words, as unsigned numbers, by powers of 16; one place of the layout at a time."""
    w = words.to(torch.int64) % (1 << 32)
    tn, tk = w.shape[:2]
    q = torch.empty((tn, 16, tk, 4, 4, 8), dtype=torch.int64, device=w.device)  # tile, row, tile, word, lane / 16, column
    lanes = w.view(tn, tk, 4, 16, 4)
    for col in range(8):
        place = 4 * (col % 2) + col // 2
        q[..., col] = (torch.div(lanes, 16 ** place, rounding_mode="floor") % 16).permute(0, 3, 1, 4, 2)
    return q.reshape(tn * 16, tk * 128)[:c["N"], :c["K"]]


def _exact_weight(q, sc, z, c):
    at = torch.div(torch.arange(c["K"], device="cuda"), c["group"], rounding_mode="floor")
    scale = sc.double()[at].t()
    return (q.double() - 8) * scale if z is None else torch.addcmul(z.double()[at].t(), q.double(), scale)


def _exact_pack(c, s):
    """Scales and codes as the 32-bit definition gives them (their roundings are part of it), the values in 64 bits."""
    w, N, K, group = s["W"].float(), c["N"], c["K"], c["group"]
    at = torch.div(torch.arange(K, device="cuda"), group, rounding_mode="floor").expand(N, K)
    n = (K + group - 1) // group
    over = lambda x, how: torch.empty((N, n), device="cuda").scatter_reduce_(1, at, x, how, include_self=False)  # noqa: E731
    if c["offset"]:
        low, high = over(w, "amin"), over(w, "amax")
        z, sc = low.to(torch.float16), ((high - low) / 15).to(torch.float16)
        q = torch.round((w - z.float().gather(1, at)) / sc.float().gather(1, at)).clamp(0, 15)
        q = q.nan_to_num(0.0)
    else:
        z, sc = None, (over(w.abs(), "amax") / 7).to(torch.float16)
        q = torch.round(w / sc.float().gather(1, at)).clamp(-8, 7).nan_to_num(0.0) + 8
    sc, z = sc.t().contiguous(), None if z is None else z.t().contiguous()
    return {"What": _exact_weight(q, sc, z, c), "s": sc.double(), "z": None if z is None else z.double()}
