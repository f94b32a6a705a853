"""Plain float64 oracle of the operators around a coupled-training layer: the product's epilogue,
the norms between blocks and the optimizer step, with their gradients.

TEST INFRASTRUCTURE ONLY, as rb_oracle.py: written from the formulas in include/rb.h, sharing no
code with the library. Every function takes arrays of any float type (widened exactly) and
returns float64, so a caller rounds or bounds as its types ask.
"""
from __future__ import annotations

import math

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


# ---------------------------------------------------------------------------------------------
# product epilogue
# ---------------------------------------------------------------------------------------------
def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activation(z, act: str):
    """(act(z), act'(z)); relu's derivative at 0 is 0."""
    z = _f(z)
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "none":
            return z, np.ones_like(z)
        if act == "relu":
            return np.where(np.isnan(z), z, np.maximum(z, 0.0)), (z > 0).astype(np.float64)
        if act == "gelu":
            cdf = 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
            return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        if act == "gelu_tanh":
            k = math.sqrt(2.0 / math.pi)
            t = np.tanh(k * (z + 0.044715 * z ** 3))
            return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 0.134145 * z * z)
        if act == "silu":
            s = _sigmoid(z)
            return z * s, s * (1.0 + z * (1.0 - s))
    raise KeyError(act)


def linear(X, What, bias=None, act: str = "none", residual=None):
    """(Y, Z): Z = X What^T + bias, Y = act(Z) + residual."""
    Z = _f(X) @ _f(What).T
    if bias is not None:
        Z = Z + _f(bias)
    Y = activation(Z, act)[0]
    return (Y if residual is None else Y + _f(residual)), Z


def linear_backward(dY, Z, act: str = "none"):
    """(dZ, db): dZ = dY act'(Z), db = its column sums."""
    dZ = _f(dY) * (1.0 if act == "none" else activation(Z, act)[1])
    return dZ, dZ.sum(axis=0)


# ---------------------------------------------------------------------------------------------
# norms between blocks
# ---------------------------------------------------------------------------------------------
def row_stats(x, kind: str, eps: float):
    """(mean, 1 / deviation) per row; the mean of an rms norm is 0, "none" has neither (0, 0)."""
    x = _f(x)
    if kind == "none":
        return np.zeros(x.shape[0]), np.zeros(x.shape[0])
    mu = x.mean(axis=1) if kind == "layer" else np.zeros(x.shape[0])
    return mu, 1.0 / np.sqrt(((x - mu[:, None]) ** 2).mean(axis=1) + eps)


def norm(x, kind: str, w, b, eps: float):
    mu, rstd = row_stats(x, kind, eps)
    y = (_f(x) - mu[:, None]) * rstd[:, None] * _f(w)
    return y if b is None else y + _f(b)


def resnorm(Y, R, w_pre, w_post=None, b_pre=None, b_post=None, gate=None, alpha=1.0, eps=1e-6, pre="rms", post="none"):
    """(S, X, stats): u = norm_post(Y), S = alpha R + gate u, X = norm_pre(S) (None for pre
    "none"); stats [M][4] = the means and 1/deviations of the post and the pre norm."""
    u = _f(Y) if post == "none" else norm(Y, post, w_post, b_post, eps)
    S = u if gate is None else _f(gate) * u
    if R is not None:
        S = alpha * _f(R) + S
    X = None if pre == "none" else norm(S, pre, w_pre, b_pre, eps)
    stats = np.stack([*row_stats(Y, post, eps), *row_stats(S, pre, eps)], axis=1)
    return S, X, stats


def norm_grad(dy, x, mu, rstd, kind: str, w):
    """(dx, dw, db) of y = norm(x) from the saved statistics."""
    dy, xh = _f(dy), (_f(x) - mu[:, None]) * rstd[:, None]
    d = dy * _f(w)
    dx = d - xh * (d * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - d.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)


def resnorm_backward(dX, dS, Y, S, stats, w_pre, w_post=None, b_post=None, gate=None, alpha=1.0, pre="rms",
                     post="none"):
    """Gradients of resnorm's inputs from those of X and S (either may be None: zero). dgate has
    the gate's shape."""
    st = _f(stats)
    T = np.zeros_like(_f(Y)) if dS is None else _f(dS)
    out = dict(dw_pre=None, db_pre=None, dw_post=None, db_post=None, dgate=None)
    if pre != "none" and dX is not None:
        dx, out["dw_pre"], out["db_pre"] = norm_grad(dX, S, st[:, 2], st[:, 3], pre, w_pre)
        T = T + dx
    out["dR"] = alpha * T
    du = T
    if gate is not None:
        u = _f(Y)
        if post != "none":
            u = (u - st[:, 0:1]) * st[:, 1:2] * _f(w_post) + (0.0 if b_post is None else _f(b_post))
        out["dgate"] = (u * T).sum(axis=0) if np.ndim(gate) == 1 else u * T
        du = _f(gate) * T
    out["dY"] = du
    if post != "none":
        out["dY"], out["dw_post"], out["db_post"] = norm_grad(du, Y, st[:, 0], st[:, 1], post, w_post)
    return out


# ---------------------------------------------------------------------------------------------
# optimizer
# ---------------------------------------------------------------------------------------------
def adamw(p, g, m, v, step: int, lr: float, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    """(p, m, v) after one step."""
    p, g = _f(p), _f(g) * grad_scale
    m, v = _f(m), _f(v)
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    hat = (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p * (1.0 - lr * weight_decay) - lr * hat, m, v


def mix32(x: int) -> int:
    """The step's hash of a 32-bit number."""
    x ^= x >> 16
    x = x * 0x9E3779B1 % (1 << 32)
    x ^= x >> 15
    x = x * 0x6A09E667 % (1 << 32)
    return x ^ (x >> 16)


def adamw_random(positions, step: int, seed: int) -> np.ndarray:
    """The 32-bit random numbers of plan positions (element i of a tensor whose first 4096-element
    chunk is number c lies at 4096 c + i)."""
    key = mix32((seed + step * 0x9E3779B1) % (1 << 32))
    return np.array([mix32((int(q) + mix32(((int(q) >> 32) + key) % (1 << 32))) % (1 << 32)) for q in positions],
                    dtype=np.int64)


E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (float("nan") if c & 127 == 127 else
                 (c & 7) / 8.0 * 2.0 ** -6 if c & 120 == 0 else (1.0 + (c & 7) / 8.0) * 2.0 ** (((c >> 3) & 15) - 7))
                 for c in range(256)])


def adamw_decode(codes, scales):
    """The values that 8-bit states stand for."""
    codes = np.asarray(codes, dtype=np.uint8)
    return E4M3[codes] / 256.0 * np.repeat(_f(scales), 256)[:codes.size]


def adamw_scales(x):
    """Per group of 256: the power of two above the largest finite magnitude, in 2^-99 .. 2^126."""
    x = np.abs(_f(x))
    x = np.where(np.isfinite(x), x, 0.0)
    top = np.array([x[i:i + 256].max() for i in range(0, x.size, 256)])
    return np.ldexp(1.0, np.frexp(np.clip(top, 2.0 ** -100, 2.0 ** 125))[1])


def adamw_grid(x, scales):
    """(a, grid): |x| in units of scale / 256 and the spacing of e4m3 numbers there."""
    a = np.abs(_f(x)) / np.repeat(scales, 256)[:np.size(x)] * 256.0
    return a, np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, -6) - 3)


# ---------------------------------------------------------------------------------------------
# gated feed-forward block
# ---------------------------------------------------------------------------------------------
def glu(X, Wg, Wu, bg=None, bu=None, act: str = "silu"):
    """(H, G, U): G = X Wg^T + bg, U = X Wu^T + bu, H = act(G) U."""
    G, U = linear(X, Wg, bg)[1], linear(X, Wu, bu)[1]
    return activation(G, act)[0] * U, G, U


def glu_backward(dH, G, U, act: str = "silu"):
    """(dG, dU, dbg, dbu) of H = act(G) U."""
    value, slope = activation(G, act)
    dG, dU = _f(dH) * _f(U) * slope, _f(dH) * value
    return dG, dU, dG.sum(axis=0), dU.sum(axis=0)


def glu_dx(dG, dU, Wg, Wu):
    return _f(dG) @ _f(Wg) + _f(dU) @ _f(Wu)


# ---------------------------------------------------------------------------------------------
# Newton-Schulz step
# ---------------------------------------------------------------------------------------------
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(u, steps: int = 5, eps: float = 1e-7):
    """X of u: its singular values taken through x -> a x + b x^3 + c x^5, `steps` times, after division by
    the Frobenius norm plus eps. From the singular value decomposition, so by another way than products."""
    u = _f(u)
    P, s, Q = np.linalg.svd(u, full_matrices=False)
    s = s / (math.sqrt((u * u).sum()) + eps)
    a, b, c = NS_COEFFICIENTS
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return (P * s) @ Q


def muon(W, G, mom, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, steps=5, eps=1e-7, grad_scale=1.0):
    """(W, mom, X) after one step; mom may be None."""
    g = _f(G) * grad_scale
    m = None if mom is None else momentum * _f(mom) + g
    u = g if m is None else g + momentum * m if nesterov else m
    X = newton_schulz(u, steps, eps)
    return (None if W is None else _f(W) * (1.0 - lr * weight_decay) - lr * scale * X), m, X


# ---------------------------------------------------------------------------------------------
# 4-bit weights with group scales
# ---------------------------------------------------------------------------------------------
def q4_quantise(W, group: int, offset: bool):
    """(codes [N][K], s [groups][N], z [groups][N] or None) of fp32 weights; s and z are fp16, every other
    step is rounded to fp32, as the definition says."""
    W = np.asarray(W, dtype=np.float32)
    N, K = W.shape
    groups = -(-K // group)
    q = np.zeros((N, K), dtype=np.int64)
    s, z = np.zeros((groups, N), dtype=np.float16), np.zeros((groups, N), dtype=np.float16)
    for g in range(groups):
        w = W[:, g * group:(g + 1) * group]
        if offset:
            lo, hi = w.min(axis=1), w.max(axis=1)
            z[g] = lo.astype(np.float16)
            s[g] = ((hi - lo) * np.float32(1 / np.float32(15))).astype(np.float16)
            d, first, last = w - z[g].astype(np.float32)[:, None], 0, 15
        else:
            s[g] = (np.abs(w).max(axis=1) * np.float32(1 / np.float32(7))).astype(np.float16)
            d, first, last = w, -8, 7
        sf = s[g].astype(np.float32)[:, None]
        with np.errstate(divide="ignore", invalid="ignore"):
            r = np.where(sf > 0, np.rint(d / sf), np.float32(0))
        q[:, g * group:(g + 1) * group] = np.clip(r, first, last).astype(np.int64) - first
    return q, s, z if offset else None


def q4_codes(q):
    """Codes [N][K] in the packed layout, [ceil(N / 16)][ceil(K / 128)][64][4] uint32, written entry by entry."""
    N, K = q.shape
    out = np.zeros((-(-N // 16), -(-K // 128), 64, 4), dtype=np.uint32)
    n, c = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    lane = 16 * (c % 32 // 8) + n % 16
    bit = 16 * (c % 2) + 4 * (c % 8 // 2)
    np.bitwise_or.at(out, (n // 16, c // 128, lane, c % 128 // 32), q.astype(np.uint32) << bit.astype(np.uint32))
    return out


def q4_values(q, s, z, group: int):
    """The weights that codes stand for."""
    at = np.arange(q.shape[1]) // group
    sc = _f(s)[at].T
    return sc * (q - 8) if z is None else sc * q + _f(z)[at].T
