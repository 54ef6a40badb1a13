"""Oracle of the feed-forward products, their gradients and the AdamW step
(numpy, fp64; the AdamW step also in the fp32 operations the device performs).

A 4-bit weight stands for the fp16 number nearest to (q - z) s.
"""
from __future__ import annotations

import math

import numpy as np

from . import dequantize

ACTIVATIONS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def weights(qweight, scales, zeros, group):
    """W_hat [rows][d] in fp64."""
    return np.asarray(dequantize(qweight, scales, zeros, group), np.float64).astype(np.float16).astype(np.float64)


def _sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


_erf = np.vectorize(math.erf, otypes=[np.float64])
_C = math.sqrt(2.0 / math.pi)


def act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    if name == "relu":
        return np.maximum(z, 0.0)
    raise ValueError(name)


def act_grad(name, z):
    if name == "none":
        return np.ones_like(z)
    if name == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    raise ValueError(name)


def preactivation(x, w, bias=None):
    z = np.asarray(x, np.float64) @ w.T
    return z if bias is None else z + np.asarray(bias, np.float64)


def linear_act(x, w, bias, residual, name):
    y = act(name, preactivation(x, w, bias))
    return y if residual is None else y + np.asarray(residual, np.float64)


def gated(x, w, bias, name):
    z = preactivation(x, w, bias)
    n = w.shape[0] // 2
    return act(name, z[:, :n]) * z[:, n:]


def linear_act_backward(x, w, bias, name, dy):
    """(dx, dz)."""
    dz = np.asarray(dy, np.float64) * act_grad(name, preactivation(x, w, bias))
    return dz @ w, dz


def gated_backward(x, w, bias, name, dy):
    z = preactivation(x, w, bias)
    n = w.shape[0] // 2
    dy = np.asarray(dy, np.float64)
    dz = np.concatenate([dy * z[:, n:] * act_grad(name, z[:, :n]), dy * act(name, z[:, :n])], axis=1)
    return dz @ w, dz


# ---------------------------------------------------------------------------
# tolerances, from the device arithmetic the header documents
# ---------------------------------------------------------------------------

U16 = 2.0 ** -11   # half a step of fp16, relative; half the smallest subnormal step is 2^-25
U32 = 2.0 ** -24
#: |act'| and |act''| are at most these for every activation (relu's jump apart)
SLOPE, BEND = 1.13, 1.2


def sum_error(x, w):
    """Bound of the error of fp32 sums x @ w.T in any order: (k + 2) 2^-24 sum |x w| (the products are exact)."""
    return (w.shape[1] + 2) * U32 * (np.abs(np.asarray(x, np.float64)) @ np.abs(w).T)


def rounded(v, err):
    """Bound after rounding v (known to err) to fp16."""
    return err + U16 * (np.abs(v) + err) + 2.0 ** -25


def act_error(z, dz):
    """Bound of the activation's and its slope's error for z known to dz: the
    evaluation itself takes at most a dozen roundings, exp2 and rcp with two
    ulps each, of terms no larger than |z| (|z| + 1) against its slope."""
    own = 32 * U32 * (1.0 + np.abs(z)) ** 2
    return SLOPE * dz + own * (1.0 + np.abs(z)), BEND * dz + own


def linear_tolerance(x, w, bias, residual, name):
    z = preactivation(x, w, bias)
    e = sum_error(x, w) + U32 * np.abs(z)
    va, _ = act_error(z, e) if name != "none" else (e, None)
    y = linear_act(x, w, bias, residual, name)
    return rounded(y, va + U32 * np.abs(y))


def gated_tolerance(x, w, bias, name):
    z = preactivation(x, w, bias)
    e = sum_error(x, w) + U32 * np.abs(z)
    n = w.shape[0] // 2
    a = act(name, z[:, :n])
    va, _ = act_error(z[:, :n], e[:, :n])
    y = a * z[:, n:]
    return rounded(y, va * (np.abs(z[:, n:]) + e[:, n:]) + np.abs(a) * e[:, n:] + U32 * np.abs(y))


def grad_tolerance(x, w, bias, name, dy, is_gated):
    """Bound of dz (before dx, which is summed from the rounded dz)."""
    z = preactivation(x, w, bias)
    e = sum_error(x, w) + U32 * np.abs(z)
    dy = np.abs(np.asarray(dy, np.float64))
    n = w.shape[0] // 2
    g, eg = (z[:, :n], e[:, :n]) if is_gated else (z, e)
    va, sa = act_error(g, eg)
    if name == "relu":  # the slope jumps where the sign of z is not known
        sa = sa + (np.abs(g) <= eg)
    s = np.abs(act_grad(name, g))
    if not is_gated:
        return rounded(dy * s, dy * sa + 2 * U32 * dy * s)
    u, eu = np.abs(z[:, n:]), e[:, n:]
    dg = dy * (s * eu + sa * (u + eu)) + 3 * U32 * dy * u * s
    a = np.abs(act(name, g))
    return np.concatenate([rounded(dy * u * s, dg), rounded(dy * a, dy * va + 2 * U32 * dy * a)], axis=1)


def input_grad_tolerance(dz, w):
    """dx for the rounded dz that the device made."""
    dz = np.asarray(dz, np.float64)
    return rounded(dz @ w, sum_error(dz, w.T.copy()))


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

def adamw(p, g, m, v, step, lr, betas, eps, weight_decay):
    """One step in fp64: (p, m, v)."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mhat, vhat = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps), m, v


def adamw_moments_f32(g, m, v, betas):
    """The moments in the device's fp32 operations, each rounded on its own."""
    f = np.float32
    b1, c1, b2, c2 = f(betas[0]), f(1.0 - betas[0]), f(betas[1]), f(1.0 - betas[1])
    g, m, v = (np.asarray(a, f) for a in (g, m, v))
    return m * b1 + g * c1, v * b2 + (g * g) * c2


E4M3 = np.array([np.ldexp(k % 8 / 8.0 + (k >= 8), max(k // 8, 1) - 7) for k in range(127)])  # codes 0 .. 126


def e4m3_codes(x):
    """e4m3 bytes nearest to x (|x| <= 448 up to rounding), ties to the even code; NaN to 0x7f."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a <= 0, 0, np.where(a >= 448, 126, code))
    return np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def e4m3_values(codes):
    codes = np.asarray(codes, np.uint8)
    mag = codes & 0x7F
    v = np.where(mag == 0x7F, np.nan, E4M3[np.minimum(mag, 126)])
    return np.where(codes & 0x80, -v, v)


def pack_moment(x, live=None):
    """Blocks of 256 fp32 values as (codes, scales) in the device's fp32 operations;
    live: values that must not become zero."""
    f = np.float32
    x = np.asarray(x, f).reshape(-1, 256)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(x).max(1)
        top = np.where(top < f(2.0 ** -100), f(0), top)
        inv = np.where(top == 0, f(0), (f(1) / top) * f(448))
        codes = e4m3_codes((x * inv[:, None]).astype(f))
    if live is not None:
        codes = np.where((codes == 0) & live.reshape(-1, 256) & (top > 0)[:, None], 1, codes).astype(np.uint8)
    return codes.reshape(-1), top * (f(1) / f(448))
