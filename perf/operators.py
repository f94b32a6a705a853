"""The operators of a training block around the residual-binarized layer, and how they are measured.

Three operators, each in its plain form (torch, 32 bits) and as a call of the library:

* linear:  Z = X What^T + b, Y = act(Z) + R, and the backward of that epilogue
           (dZ = dY act'(Z), db = the column sums of dZ);
* resnorm: u = norm_post(Y), S = alpha R + gate u, X = norm_pre(S), and its backward;
* adamw:   one optimizer step over many tensors, states in 32 bits or in 8.

``own`` selects the form. Inputs are seeded; effective weights are sums of two sign planes with row
and column scales, as the layer's derivation gives them.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
CHUNK = 4096   # elements of one tensor that one optimizer block takes; random positions count in these
GROUP = 256    # elements that share a scale in the 8-bit states
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _linear(M, N, K, dt, act, bias, res, y_dt, save_z, pad=0):
    return dict(op="linear", M=M, N=N, K=K, dt=dt, act=act, bias=bias, res=res, y_dt=y_dt, save_z=save_z, pad=pad)


def _linear_bwd(M, N, dt, act, bias, dy_dt):
    return dict(op="linear_bwd", M=M, N=N, dt=dt, act=act, bias=bias, dy_dt=dy_dt)


def _resnorm(back, M, D, dt, s_dt, post, pre, gate, bias):
    return dict(op="resnorm_bwd" if back else "resnorm", M=M, D=D, dt=dt, s_dt=s_dt, post=post, pre=pre, gate=gate,
                bias=bias)


def _adamw(bits, p_dt, g_dt, layers, N, K, planes, scale):
    return dict(op="adamw", bits=bits, p_dt=p_dt, g_dt=g_dt, layers=layers, N=N, K=K, planes=planes, scale=scale)


def listed():
    return [
        # one token through the 4096 x 4096 layer with its residual: a decode step, latency
        dict(_linear(1, 4096, 4096, "f16", "none", False, True, "f16", False), name="linear 1 token 4096x4096"),
        # a short ragged batch on an odd layer whose rows are not 16-byte aligned
        dict(_linear(61, 1027, 1411, "bf16", "gelu", True, False, "f32", True), name="linear ragged 61x1027x1411"),
        # 2048 tokens into the 11008-wide half of the MLP: activation, pre-activation kept for training
        dict(_linear(2048, 11008, 4096, "bf16", "silu", True, False, "bf16", True), name="linear up 2048 tokens"),
        # ... and back out of it, added to an fp32 residual stream
        dict(_linear(2048, 4096, 11008, "bf16", "none", True, True, "f32", False), name="linear down 2048 tokens"),
        # the epilogue's backward at the same MLP width
        dict(_linear_bwd(2048, 11008, "bf16", "silu", True, "bf16"), name="linear backward 2048 tokens"),
        # one token between two blocks: latency
        dict(_resnorm(False, 1, 4096, "f16", "f16", "rms", "rms", "none", False), name="resnorm 1 token"),
        # a training batch: fp32 stream, learned gate per channel
        dict(_resnorm(False, 2048, 4096, "bf16", "f32", "rms", "rms", "channel", False), name="resnorm 2048x4096"),
        dict(_resnorm(True, 2048, 4096, "bf16", "f32", "rms", "rms", "channel", False),
             name="resnorm backward 2048x4096"),
        # odd rows and an odd width, centred norms with biases, a gate for each element
        dict(_resnorm(True, 1537, 8191, "bf16", "bf16", "layer", "layer", "element", True),
             name="resnorm backward odd 1537x8191"),
        # the scales and weight of one small layer: launch latency
        dict(_adamw(32, "f32", "f32", 1, 256, 512, 1, False), name="adamw one small layer"),
        # the three MLP layers, 135 M shared weights with their scales, 32-bit states
        dict(_adamw(32, "f32", "f32", 3, 4096, 11008, 2, True), name="adamw mlp 32-bit"),
        # the same with 8-bit states
        dict(_adamw(8, "f32", "f32", 3, 4096, 11008, 2, True), name="adamw mlp 8-bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm; half of them multiples of 160, the others as they fall."""
    n = _log(rng, lo, hi)
    return n // 160 * 160 if n >= 160 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "resnorm", "resnorm_bwd", "adamw", "adamw"])
    dt = rng.choice(["bf16", "f16"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 4096), _size(rng, 200, 11008), _size(rng, 200, 11008)
            if M * N * K <= 2048 * 4096 * 11008:
                break
        return _linear(M, N, K, dt, rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.6,
                       rng.random() < 0.5, rng.choice([dt, "f32"]), rng.random() < 0.4, rng.choice([0, 0, 8, 3]))
    if op == "linear_bwd":
        M, N = _log(rng, 1, 4096), _size(rng, 200, 11008)
        return _linear_bwd(M, N, dt, rng.choice(["relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.8,
                           rng.choice([dt, "f32"]))
    if op in ("resnorm", "resnorm_bwd"):
        M, D = _log(rng, 1, 8192), _size(rng, 100, 8192)
        return _resnorm(op == "resnorm_bwd", M, D, dt, rng.choice([dt, "f32"]), rng.choice(["none", "rms", "layer"]),
                        rng.choice(["rms", "layer"]), rng.choice(["none", "channel", "element"]), rng.random() < 0.5)
    layers = _log(rng, 1, 64)
    while True:
        N, K = _size(rng, 64, 11008), _size(rng, 64, 11008)
        if layers * N * K <= 3 * 4096 * 11008:
            break
    return _adamw(rng.choice([8, 32]), *rng.choice([("f32", "f32"), ("f32", "f32"), ("f32", dt), (dt, dt)]), layers, N, K,
                  rng.choice([1, 2, 3, 4]), rng.random() < 0.5)


def _rows(n):
    return (n + GROUP - 1) // GROUP


def _adamw_layout(c):
    """(length, decay) of every tensor of a case: the layers' weights, then their scales."""
    weights = [(c["N"] * c["K"], DECAY)] * c["layers"]
    scales = [(c["planes"] * c["N"], 0.0), (c["planes"] * c["K"], 0.0)] * c["layers"]
    return weights + scales


def work(c):
    """Each input read once, each output written once."""
    if c["op"] == "linear":
        M, N, K, e, y = c["M"], c["N"], c["K"], SIZE[c["dt"]], SIZE[c["y_dt"]]
        b = (M * K + N * K) * e + M * N * y * (1 + c["res"]) + M * N * e * c["save_z"] + 4 * N * c["bias"]
        return {"bytes": b, "flops": 2 * M * N * K}
    if c["op"] == "linear_bwd":
        M, N, e = c["M"], c["N"], SIZE[c["dt"]]
        return {"bytes": M * N * (SIZE[c["dy_dt"]] + 2 * e) + 4 * N * c["bias"], "flops": 10 * M * N}
    if c["op"] in ("resnorm", "resnorm_bwd"):
        M, D, e, s = c["M"], c["D"], SIZE[c["dt"]], SIZE[c["s_dt"]]
        vec = 4 * D * ((1 + c["bias"]) * ((c["post"] != "none") + 1) + (c["gate"] == "channel"))
        el = c["gate"] == "element"
        if c["op"] == "resnorm":
            return {"bytes": M * D * (2 * e + 2 * s + e * el) + vec + 16 * M, "flops": 10 * M * D}
        return {"bytes": M * D * (3 * e + 3 * s + 2 * e * el) + 2 * vec + 16 * M, "flops": 25 * M * D}
    n = sum(t[0] for t in _adamw_layout(c))
    p, g = SIZE[c["p_dt"]], SIZE[c["g_dt"]]
    state = 16 * n if c["bits"] == 32 else 4 * n + 16 * sum(_rows(t[0]) for t in _adamw_layout(c))
    return {"bytes": n * (2 * p + g) + state, "flops": 15 * n}


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


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "linear":
        M, N, K, dt = c["M"], c["N"], c["K"], DT[c["dt"]]
        s["X"] = _normal(g, (M, K), dt, pad=c["pad"])
        s["What"] = _effective_weight(g, N, K, dt, c["pad"])
        s["bias"] = _normal(g, (N,), torch.float32, 0.1) if c["bias"] else None
        s["R"] = _normal(g, (M, N), DT[c["y_dt"]]) if c["res"] else None
        s["Y"] = torch.empty((M, N), dtype=DT[c["y_dt"]], device="cuda")
        s["Z"] = torch.empty((M, N), dtype=dt, device="cuda") if c["save_z"] else None
    elif c["op"] == "linear_bwd":
        M, N, dt = c["M"], c["N"], DT[c["dt"]]
        s["dY"] = _normal(g, (M, N), DT[c["dy_dt"]], 0.01)
        s["Z"] = _normal(g, (M, N), dt, 1.5)
        s["dZ"] = torch.empty((M, N), dtype=dt, device="cuda")
        s["db"] = torch.empty(N, device="cuda") if c["bias"] else None
    elif c["op"] in ("resnorm", "resnorm_bwd"):
        _prepare_resnorm(c, g, s)
    else:
        _prepare_adamw(c, g, s)
    return s


def _prepare_resnorm(c, g, s):
    M, D, dt, sdt = c["M"], c["D"], DT[c["dt"]], DT[c["s_dt"]]
    post = c["post"] != "none"
    s["Y"] = _normal(g, (M, D), dt, 0.7)
    s["w_pre"] = _vector(g, D, 0.5, 1.5)
    s["w_post"] = _vector(g, D, 0.5, 1.5) if post else None
    s["b_pre"] = _normal(g, (D,), torch.float32, 0.1) if c["bias"] else None
    s["b_post"] = _normal(g, (D,), torch.float32, 0.1) if c["bias"] and post else None
    s["gate"] = {"none": lambda: None, "channel": lambda: _vector(g, D, -0.5, 1.0),
                 "element": lambda: _normal(g, (M, D), dt, 0.5)}[c["gate"]]()
    s["alpha"] = 0.9
    if c["op"] == "resnorm":
        s["R"] = _normal(g, (M, D), sdt)
        s["S"], s["X"] = torch.empty((M, D), dtype=sdt, device="cuda"), torch.empty((M, D), dtype=dt, device="cuda")
        s["stats"] = torch.empty((M, 4), device="cuda")
        return
    # what the forward left: the stream S and the statistics (mean, 1/deviation) of both norms
    s["S"] = _normal(g, (M, D), sdt, 1.3)
    s["dX"] = _normal(g, (M, D), dt, 0.01)
    s["dS"] = _normal(g, (M, D), sdt, 0.01)
    stats = torch.zeros((M, 4), device="cuda")
    for k, kind, x in ((0, c["post"], s["Y"]), (2, c["pre"], s["S"])):
        if kind != "none":
            x = x.double()
            mu = x.mean(1) if kind == "layer" else torch.zeros(M, dtype=torch.float64, device="cuda")
            stats[:, k] = mu.float()
            stats[:, k + 1] = ((x - mu[:, None]).square().mean(1) + EPS).rsqrt().float()
    s["stats"] = stats
    s["dY"], s["dR"] = torch.empty((M, D), dtype=dt, device="cuda"), torch.empty((M, D), dtype=sdt, device="cuda")


def _prepare_adamw(c, g, s):
    """The tensors lie in one buffer of each kind, every tensor from a multiple of GROUP elements."""
    layout = _adamw_layout(c)
    rows = [_rows(n) for n, _ in layout]
    first, at, chunk, row_pos = [], 0, 0, []
    for (n, _), r in zip(layout, rows):
        first.append(at * GROUP)
        row_pos.append(torch.arange(r, dtype=torch.int64) * GROUP + chunk * CHUNK)
        at += r
        chunk += (n + CHUNK - 1) // CHUNK
    s["row_pos"] = torch.cat(row_pos).cuda()  # where each row of GROUP elements lies in the step's random sequence
    s["decayed"] = sum(rows[: c["layers"]]) * GROUP  # the weights, which decay, come first
    total = at * GROUP
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for (n, _), o in zip(layout, first):
        live[o:o + n] = True
    p = torch.randn(total, generator=g, device="cuda").mul_(0.02).mul_(live).to(DT[c["p_dt"]])
    # a training run some steps in: gradients of very different sizes, a few entries never touched
    size = torch.exp(torch.randn((at, 1), generator=g, device="cuda") - 8)
    touched = (torch.rand(total, generator=g, device="cuda") > 0.02).mul_(live)
    grad = torch.randn((at, GROUP), generator=g, device="cuda").mul_(size).reshape(-1).mul_(touched).to(DT[c["g_dt"]])
    m = torch.randn((at, GROUP), generator=g, device="cuda").mul_(size * 0.3).mul_(touched.reshape(at, GROUP))
    r = (torch.rand((at, GROUP), generator=g, device="cuda") + 0.5).mul_(size).mul_(touched.reshape(at, GROUP))
    s["p"], s["g"] = p, grad
    s["grad_scale"] = torch.rand(1, generator=g, device="cuda").mul_(0.5).add_(0.5) if c["scale"] else None
    s["step"], s["seed"] = 10, int(torch.randint(1 << 31, (1,), generator=g, device="cuda"))
    if c["bits"] == 32:
        s["m"], s["v"] = m.reshape(-1), r.square().reshape(-1)
    else:
        for name, x in (("m", m), ("v", r)):
            scale = torch.exp2(torch.floor(torch.log2(x.abs().amax(1).clamp_min(2.0 ** -100))) + 1)
            s[name] = (x / scale[:, None] * 256).to(torch.float8_e4m3fn).reshape(-1)
            s[name + "_scale"] = scale
    if own:  # the table of tensors that a training program builds once
        import residual_binarized_weight_amd as rb
        parts = lambda t: [t[o:o + n] for (n, _), o in zip(layout, first)]  # noqa: E731
        more = {}
        if c["bits"] == 8:
            at_row = [o // GROUP for o in first]
            more = {k: [s[k][o:o + r] for o, r in zip(at_row, rows)] for k in ("m_scale", "v_scale")}
        s["plan"] = rb.adamw_plan(parts(s["p"]), parts(s["g"]), state_bits=c["bits"], m=parts(s["m"]), v=parts(s["v"]),
                                  weight_decay=[w for _, w in layout], **more)


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import residual_binarized_weight_amd as rb
    c = s["c"]
    if c["op"] == "linear":
        Y, Z = rb.qat_linear(s["X"], s["What"], bias=s["bias"], act=c["act"], residual=s["R"], Y=s["Y"], Z=s["Z"])
        return {"Y": Y, "Z": Z}
    if c["op"] == "linear_bwd":
        dZ, db = rb.qat_linear_backward(s["dY"], s["Z"], act=c["act"], dZ=s["dZ"], bias=c["bias"], db=s["db"])
        return {"dZ": dZ, "db": db}
    if c["op"] == "resnorm":
        S, X, stats = rb.resnorm_forward(s["Y"], s["R"], s["w_pre"], w_post=s["w_post"], b_pre=s["b_pre"],
                                         b_post=s["b_post"], gate=s["gate"], alpha=s["alpha"], eps=EPS, pre=c["pre"],
                                         post=c["post"], S=s["S"], X=s["X"], stats=s["stats"])
        return {"S": S, "X": X, "stats": stats}
    if c["op"] == "resnorm_bwd":
        return rb.resnorm_backward(s["dX"], s["dS"], s["Y"], s["S"], s["stats"], s["w_pre"], w_post=s["w_post"],
                                   b_post=s["b_post"], gate=s["gate"], alpha=s["alpha"], pre=c["pre"], post=c["post"],
                                   bias=c["bias"], dY=s["dY"], dR=s["dR"])
    s["step"] += 1
    rb.adamw_step(s["plan"], s["step"], LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, grad_scale=s["grad_scale"],
                  seed=s["seed"])
    return {k: s[k] for k in ("p", "m", "v", "m_scale", "v_scale") if k in s}


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


def _norm(x, kind, w, b):
    """(normed, mean, 1/deviation) of the rows of x."""
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = ((x - mu).square().mean(1, keepdim=True) + EPS).rsqrt()
    y = (x - mu) * rstd * w
    return (y if b is None else y + b), mu, rstd


def _norm_grad(dy, x, kind, w, mu, rstd):
    """(dx, dw, db) of the rows' norm."""
    xh, d = (x - mu) * rstd, dy * w
    dx = d - xh * (d * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - d.mean(1, keepdim=True)
    return dx * rstd, (dy * xh).sum(0), dy.sum(0)


def _run_plain(s):
    c = s["c"]
    if c["op"] == "linear":
        z = s["X"].float() @ s["What"].float().t()
        if c["bias"]:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if c["res"]:
            y = y + s["R"].float()
        return {"Y": y.to(DT[c["y_dt"]]), "Z": z.to(DT[c["dt"]]) if c["save_z"] else None}
    if c["op"] == "linear_bwd":
        dz = s["dY"].float() * _act_slope(s["Z"].float(), c["act"])
        return {"dZ": dz.to(DT[c["dt"]]), "db": dz.sum(0) if c["bias"] else None}
    if c["op"] == "resnorm":
        u = s["Y"].float()
        mu_post = rstd_post = torch.zeros_like(u[:, :1])
        if c["post"] != "none":
            u, mu_post, rstd_post = _norm(u, c["post"], s["w_post"], s["b_post"])
        if c["gate"] != "none":
            u = s["gate"].float() * u
        stream = s["alpha"] * s["R"].float() + u
        x, mu_pre, rstd_pre = _norm(stream, c["pre"], s["w_pre"], s["b_pre"])
        return {"S": stream.to(DT[c["s_dt"]]), "X": x.to(DT[c["dt"]]),
                "stats": torch.cat([mu_post, rstd_post, mu_pre, rstd_pre], 1)}
    if c["op"] == "resnorm_bwd":
        return _plain_resnorm_bwd(s)
    return _plain_adamw(s)


def _plain_resnorm_bwd(s):
    c, stats = s["c"], s["stats"]
    d, dw_pre, db_pre = _norm_grad(s["dX"].float(), s["S"].float(), c["pre"], s["w_pre"], stats[:, 2:3], stats[:, 3:4])
    d = d + s["dS"].float()
    out = {"dR": (s["alpha"] * d).to(DT[c["s_dt"]]), "dw_pre": dw_pre, "db_pre": db_pre if c["bias"] else None,
           "dgate": None, "dw_post": None, "db_post": None}
    y = s["Y"].float()
    if c["gate"] != "none":
        u = y
        if c["post"] != "none":
            u = (y - stats[:, 0:1]) * stats[:, 1:2] * s["w_post"]
            u = u if s["b_post"] is None else u + s["b_post"]
        out["dgate"] = (u * d).sum(0) if c["gate"] == "channel" else (u * d).to(DT[c["dt"]])
        d = s["gate"].float() * d
    if c["post"] != "none":
        d, out["dw_post"], db_post = _norm_grad(d, y, c["post"], s["w_post"], stats[:, 0:1], stats[:, 1:2])
        out["db_post"] = db_post if c["bias"] else None
    out["dY"] = d.to(DT[c["dt"]])
    return out


def _mix(x):
    """A bijective mix of 32-bit numbers (held in int64): xor-shifts and products with odd constants."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(s):
    """One 32-bit number for each element, in rows of GROUP: a hash of its position, the seed and the step."""
    key = _mix(torch.tensor((s["seed"] + s["step"] * 0x9E3779B1) & 0xFFFFFFFF, device="cuda"))
    row = (_mix(((s["row_pos"] >> 32) + key) & 0xFFFFFFFF) + s["row_pos"]) & 0xFFFFFFFF
    return _mix((row[:, None] + torch.arange(GROUP, device="cuda")) & 0xFFFFFFFF)


def _decode(codes, scale):
    return codes.float().reshape(-1, GROUP) * (2.0 ** -8) * scale[:, None]


def _encode(x, low, sixteen):
    """(e4m3 values, scales) of rows of GROUP values: each row's scale is the power of two above its largest
    finite magnitude and stands for 256; the 20 fraction bits that do not fit are rounded up where 16 random
    bits say so. What is not finite becomes NaN; ``low`` is the smallest code that a nonzero value takes."""
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0).amax(1).clamp(2.0 ** -100, 2.0 ** 125)
    bits = (top.view(torch.int32) & 0x7F800000) + 0x00800000
    y = x.abs() * ((254 << 23) - bits).view(torch.float32)[:, None] * 2.0 ** -112
    code = (y.view(torch.int32).to(torch.int64) + sixteen * 16 + 8) >> 20
    code = torch.where(x == 0, 0, code.clamp(low, 0x7E))
    code = torch.where(fine, code, 0x7F) | torch.where(torch.signbit(x), 0x80, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn).reshape(-1), bits.view(torch.float32)


def _plain_adamw(s):
    c = s["c"]
    s["step"] += 1
    g = s["g"].float()
    if s["grad_scale"] is not None:
        g = g * s["grad_scale"]
    small = c["bits"] == 8
    m = _decode(s["m"], s["m_scale"]).reshape(-1) if small else s["m"]
    v = _decode(s["v"], s["v_scale"]).square().reshape(-1) if small else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    r = torch.sqrt(v)
    d = (LR / (1 - BETA1 ** s["step"])) * (m / (r * (1 / math.sqrt(1 - BETA2 ** s["step"])) + ADAM_EPS))
    n = s["decayed"]
    s["p"][:n] = s["p"][:n].float() * (1 - LR * DECAY) - d[:n]
    s["p"][n:] = s["p"][n:].float() - d[n:]
    if not small:
        s["m"], s["v"] = m, v
        return {k: s[k] for k in ("p", "m", "v")}
    h = _random(s)
    s["m"], s["m_scale"] = _encode(m.reshape(-1, GROUP), 0, h & 0xFFFF)
    s["v"], s["v_scale"] = _encode(r.reshape(-1, GROUP), 1, h >> 16)
    return {k: s[k] for k in ("p", "m", "v", "m_scale", "v_scale")}


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
    if c["op"] == "linear":
        z = torch.mm(f["X"], f["What"].t().contiguous())
        z = z if f["bias"] is None else z + f["bias"]
        y = _exact_act(z, c["act"])[0]
        return {"Y": y if f["R"] is None else y + f["R"], "Z": z if c["save_z"] else None}
    if c["op"] == "linear_bwd":
        dz = f["dY"] * _exact_act(f["Z"], c["act"])[1]
        return {"dZ": dz, "db": torch.mv(dz.t(), torch.ones_like(dz[:, 0])) if c["bias"] else None}
    if c["op"] == "resnorm":
        return _exact_resnorm(c, f)
    if c["op"] == "resnorm_bwd":
        return _exact_resnorm_bwd(c, f)
    return _exact_adamw(c, s)


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


def _exact_hat(x, kind):
    if kind == "layer":
        var, mu = torch.var_mean(x, 1, correction=0, keepdim=True)
    else:
        var, mu = (x * x).sum(1, keepdim=True) / x.shape[1], torch.zeros_like(x[:, :1])
    rstd = 1 / torch.sqrt(var + EPS)
    return (x - mu) * rstd, mu, rstd


def _exact_resnorm(c, f):
    u, none = f["Y"], torch.zeros_like(f["Y"][:, :1])
    st = [none, none]
    if c["post"] != "none":
        u, *st = _exact_hat(u, c["post"])
        u = torch.addcmul(f["b_post"] if c["bias"] else torch.zeros_like(u[0]), u, f["w_post"])
    stream = f["R"] * f["alpha"] + (u if f["gate"] is None else u * f["gate"])
    h, *st2 = _exact_hat(stream, c["pre"])
    return {"S": stream, "X": h * f["w_pre"] + (f["b_pre"] if c["bias"] else 0), "stats": torch.cat(st + st2, 1)}


def _exact_resnorm_bwd(c, f):
    """Each norm's Jacobian, applied as a projection: off the ones (centred norms), and off the normed row."""
    def back(d, h, kind, rstd):
        n = d.shape[1]
        if kind == "layer":
            d = d - d.sum(1, keepdim=True) / n
        return (d - h * torch.linalg.vecdot(d, h)[:, None] / n) * rstd

    st = f["stats"].unbind(1)
    h = (f["S"] - st[2][:, None]) * st[3][:, None]
    t = back(f["dX"] * f["w_pre"], h, c["pre"], st[3][:, None]) + f["dS"]
    out = {"dR": t * f["alpha"], "dw_pre": (f["dX"] * h).sum(0), "db_pre": f["dX"].sum(0) if c["bias"] else None}
    post = c["post"] != "none"
    yh = (f["Y"] - st[0][:, None]) * st[1][:, None] if post else f["Y"]
    u = yh * f["w_post"] if post else yh
    u = u + f["b_post"] if f["b_post"] is not None else u
    out["dgate"] = {"none": lambda: None, "channel": lambda: (t * u).sum(0), "element": lambda: t * u}[c["gate"]]()
    du = t if f["gate"] is None else t * f["gate"]
    out["dw_post"] = (du * yh).sum(0) if post else None
    out["db_post"] = du.sum(0) if post and c["bias"] else None
    out["dY"] = back(du * f["w_post"], yh, c["post"], st[1][:, None]) if post else du
    return out


def _exact_round(x, low, uniform):
    """Stochastic rounding to the e4m3 grid times each row's power of two; (values on the grid, scales)."""
    top = x.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
    scale = torch.exp2(torch.frexp(top)[1].double())
    a = x.abs() / scale * 256
    # normal numbers hold 4 significant bits; below 2^-6 the grid stays at 2^-9
    grid = torch.exp2((torch.frexp(a)[1] - 1).clamp_min(-6).double() - 3)
    q = torch.floor(a / grid + uniform) * grid
    q = torch.where(x == 0, 0, q.clamp_min(low))
    return (torch.sign(x) * q).reshape(-1), scale.reshape(-1)


def _exact_adamw(c, s):
    t = s["step"] + 1
    g = s["g"].double() * (1 if s["grad_scale"] is None else s["grad_scale"].double())
    m, r2 = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = (m.reshape(-1, GROUP) * s["m_scale"].double()[:, None] / 256).reshape(-1)
        r2 = (r2.reshape(-1, GROUP) * s["v_scale"].double()[:, None] / 256).reshape(-1) ** 2
    m, r2 = torch.lerp(g, m, BETA1), torch.lerp(g * g, r2, BETA2)
    decay = torch.ones_like(m)
    decay[: s["decayed"]] -= LR * DECAY
    hat = m / (1 - BETA1 ** t) / (torch.sqrt(r2 / (1 - BETA2 ** t)) + ADAM_EPS)
    out = {"p": s["p"].double() * decay - LR * hat, "m": m, "v": r2}
    if c["bits"] == 32:
        return out

    def scramble(x):  # the same 32-bit mix, as remainders
        for shift, factor in ((16, 2654435761), (15, 1779033703)):
            x = torch.bitwise_xor(x, torch.div(x, 1 << shift, rounding_mode="floor"))
            low, high = x % 65536, torch.div(x, 65536, rounding_mode="floor")
            x = (low * factor + (high * factor % 65536) * 65536) % (1 << 32)
        return torch.bitwise_xor(x, torch.div(x, 65536, rounding_mode="floor"))

    pos = s["row_pos"][:, None] + torch.arange(GROUP, device="cuda")
    key = scramble(torch.tensor([(s["seed"] + t * 2654435761) % (1 << 32)], device="cuda"))
    high = scramble((torch.div(pos[:, :1], 1 << 32, rounding_mode="floor") + key) % (1 << 32))
    h = scramble((high + pos) % (1 << 32))
    out["m"], out["m_scale"] = _exact_round(m.reshape(-1, GROUP), 0.0, (h % 65536 + 0.5) / 65536)
    low = 2.0 ** -9
    out["v"], out["v_scale"] = _exact_round(r2.sqrt().reshape(-1, GROUP), low,
                                            (torch.div(h, 65536, rounding_mode="floor") + 0.5) / 65536)
    return out
