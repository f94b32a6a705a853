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
