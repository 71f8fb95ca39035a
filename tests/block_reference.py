"""Block norms, products with an epilogue and their gradients in 64 bits (numpy), with bounds on
what a computation in binary32 may differ by."""
import math

import numpy as np
import torch
from scipy.special import erf, erfc

U = 2.0 ** -24   # half a unit in the last place of binary32, relative
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a unit in the last place of each type, relative, and half the smallest step of the type
HALF = {d: torch.finfo(t).eps / 2 for d, t in TYPES.items()}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
C = 2 * math.sqrt(2 / math.pi)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v < 0, e, 1.0) / (1 + e)


def act(v, a):
    if a == "relu":
        return np.where(v < 0, 0.0, v)
    if a == "gelu":
        return v * 0.5 * erfc(-v / math.sqrt(2))
    if a == "gelu_tanh":
        return v * _sigmoid(C * (v + 0.044715 * v ** 3))
    if a == "silu":
        return v * _sigmoid(v)
    return v


def slope(v, a):
    if a == "relu":
        return (v > 0).astype(v.dtype)
    if a == "gelu":
        return 0.5 * (1 + erf(v / math.sqrt(2))) + v * np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if a == "gelu_tanh":
        z = C * (v + 0.044715 * v ** 3)
        return _sigmoid(z) + v * _sigmoid(z) * _sigmoid(-z) * C * (1 + 3 * 0.044715 * v * v)
    if a == "silu":
        return _sigmoid(v) + v * _sigmoid(v) * _sigmoid(-v)
    return np.ones_like(v)


# Activations in binary32: exponents of up to 87 are rounded (87 U each, once for the square and once
# for the product with log2 e), the fit, the reciprocal and a few products add up to less than 20 U.
ACT = 200 * U
# Derivatives cancel at most against terms of size 1 + |v| where e^-|v| is not yet small: sizes of
# up to 2 in units of their terms.
SLOPE = 400 * U
STEEPEST = 1.13  # the largest slope of the activations here


def rms(v, eps):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


# A row's sum of squares: at most 32 terms in a thread, 6 and 16 joins, all terms positive, so 54
# roundings of at most U; its root has half of that; mean, root, reciprocal and the products around
# it add 8.
NORM = 40 * U


def block_norm(r, y=None, post=False, post_weight=None, gate=None, scale=1.0, weight=None, eps=1e-6):
    """(new residual, its bound, output, its bound) before any rounding to a type."""
    new, bound = r, np.zeros_like(r)
    if y is not None:
        u = y
        if post:
            u = y / rms(y, eps) * (1.0 if post_weight is None else post_weight)
        add = scale * u * (1.0 if gate is None else gate)
        new = r + add
        bound = np.abs(add) * (NORM + 3 * U) + np.abs(new) * U
    s = rms(new, eps)
    w = np.ones(r.shape[1]) if weight is None else weight
    out = new / s * w
    # the root's relative change is at most that of the row's norm
    moved = np.sqrt((bound ** 2).mean(axis=1, keepdims=True)) / s
    return new, bound, out, bound / s * np.abs(w) + np.abs(out) * (NORM + moved)


# Sums of signed terms along a row: 54 roundings, and those of the terms; sums over rows: at most
# ceil(rows / 512) + 3 + 32 + 16 additions (the tests' rows: below 100 in all).
SUM = 100 * U


def block_norm_backward(d_out, d_new, r, y=None, post=False, post_weight=None, gate=None, scale=1.0, weight=None, eps=1e-6):
    """{name: (gradient, bound)}; gate of one dimension: summed over rows."""
    w = np.ones(r.shape[1]) if weight is None else weight
    s = 1 / rms(r, eps)
    dn = d_out * w
    along = s * s * (dn * r).mean(axis=1, keepdims=True)
    size = s * s * np.abs(dn * r).mean(axis=1, keepdims=True)
    d_r = d_new + s * (dn - r * along)
    e_r = SUM * (np.abs(d_new) + s * (np.abs(dn) + np.abs(r) * size))
    got = {"d_residual": (d_r, e_r),
           "d_weight": ((d_out * r * s).sum(axis=0), 2 * SUM * np.abs(d_out * r * s).sum(axis=0))}
    if y is None:
        return got
    z = 1 / rms(y, eps) if post else 1.0
    pw = np.ones(r.shape[1]) if post_weight is None else post_weight
    j, f = y * z, 1.0 if gate is None else gate
    if gate is not None:
        d_gate, e = scale * d_r * j * pw, np.abs(scale * j * pw) * (e_r + (NORM + 6 * U) * np.abs(d_r))
        got["d_gate"] = (d_gate, e) if gate.ndim == 2 else (d_gate.sum(axis=0), (e + SUM * np.abs(d_gate)).sum(axis=0))
    g = scale * d_r * f
    e_g = np.abs(scale * f) * (e_r + 3 * U * np.abs(d_r))
    if not post:
        got["d_y"] = (g, e_g)
        return got
    got["d_post_weight"] = ((g * j).sum(axis=0), (e_g * np.abs(j) + 2 * SUM * np.abs(g * j)).sum(axis=0))
    p, e_p = g * pw, np.abs(pw) * e_g + 2 * U * np.abs(g * pw)
    back = z * z * (p * y).mean(axis=1, keepdims=True)
    e_back = z * z * (e_p * np.abs(y) + SUM * np.abs(p * y)).mean(axis=1, keepdims=True)
    got["d_y"] = (z * (p - y * back), z * (e_p + np.abs(y) * e_back + (NORM + 6 * U) * (np.abs(p) + np.abs(y * back))))
    return got


# A product over k in binary32: each matrix instruction adds 16 or 32 products to the accumulator, and joins
# of partial sums follow; every one of those rounds to at most 2^-23 of the size of the terms.
def product(a, b):
    """(a b^T, bound)"""
    steps = a.shape[1] / 8 + 16
    return a @ b.T, np.abs(a) @ np.abs(b).T * steps * 2.0 ** -23


def linear(x, w, bias=None, a="none", residual=None):
    """(pre, bound, out, bound) before rounding to a type."""
    pre, e = product(x, w)
    if bias is not None:
        pre = pre + bias
        e = e + U * np.abs(pre)
    out = act(pre, a)
    e_out = STEEPEST * e + ACT * np.abs(out) + U * np.abs(pre) * (a != "none")
    if residual is not None:
        out = out + residual
        e_out = e_out + U * np.abs(out)
    return pre, e, out, e_out


def close(got, want, bound, dtype, what=""):
    """got is want within bound and one rounding to the type."""
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    limit = bound + (np.abs(want) + bound) * HALF[dtype] + TINY[dtype]
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off, the worst by "
                           f"{np.nanmax(np.abs(got - want) / limit)} of its bound, at {np.argwhere(bad)[0]}")


def rounded(a, dtype):
    """A tensor of the type on the CPU and its values in 64 bits."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype])
    return t, t.double().numpy()
