"""Oracle of the mixture-of-experts operators and the distillation loss (numpy,
fp64), with the bounds that follow from the device's documented arithmetic."""
from __future__ import annotations

import numpy as np

from . import block
from .block import U32, rounded, sum_error

#: half a step relative to the value, and half of the smallest subnormal step
HALF_STEP = {"fp32": (2.0 ** -24, 2.0 ** -150), "fp16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}


def stored(v, err, kind):
    """Bound after rounding v (known to err) to a type."""
    u, tiny = HALF_STEP[kind]
    return err + u * (np.abs(v) + err) + tiny


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------

def route(logits, k, normalize):
    """(ids [M][k], weights [M][k]) of logits [M][E]."""
    x = np.asarray(logits, np.float64)
    ids = np.full((len(x), k), -1, np.int64)
    w = np.zeros((len(x), k))
    for m, row in enumerate(x):
        live = np.flatnonzero(row > -np.inf)
        pick = live[np.argsort(-row[live], kind="stable")][:k]
        ids[m, :len(pick)] = pick
        if len(pick):
            with np.errstate(invalid="ignore"):
                e = np.exp(row - row[pick[0]])
            total = e[pick].sum() if normalize else e[live].sum()
            w[m, :len(pick)] = np.nan if np.isnan(row).any() else e[pick] / total
    return ids, w


def route_tolerance(logits, ids, w, normalize):
    """exp2 within 3 ulps (0 below 2^-126) of an argument rounded twice, fp32 sums over at most E experts."""
    x = np.asarray(logits, np.float64)
    E = x.shape[1]
    top = np.where(np.isfinite(x).any(1), np.max(np.where(np.isfinite(x), x, -np.inf), 1, initial=-1e30), 0.0)
    span = top[:, None] - np.take_along_axis(np.where(np.isfinite(x), x, 0.0), np.maximum(ids, 0), 1)
    return np.abs(w) * U32 * (2 * np.abs(span) + E + 16) + 2.0 ** -126


def tables(ids, E):
    """(offsets [E + 1], order [R], place [R])."""
    flat = np.asarray(ids).reshape(-1)
    live = (flat >= 0) & (flat < E)
    key = np.where(live, flat, E)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(flat))
    n = int(live.sum())
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return offsets, np.where(np.arange(len(flat)) < n, order, -1), np.where(live, place, -1)


def route_backward(logits, ids, w, dw, normalize):
    """(dlogits, its bound before rounding) for the ids and weights that the forward call returned."""
    x = np.asarray(logits, np.float64)
    M, E = x.shape
    k = ids.shape[1]
    live = ids >= 0
    w, dw = np.where(live, w, 0.0), np.where(live, dw, 0.0)
    inner = (w * dw).sum(1, keepdims=True)
    e_inner = (k + 2) * U32 * np.abs(w * dw).sum(1, keepdims=True)
    out, err = np.zeros((M, E)), np.zeros((M, E))
    if not normalize:
        for m in range(M):
            if (x[m] > -np.inf).any():
                t = x[m] - x[m].max()
                p = np.exp(t) / np.exp(t).sum()
                out[m] = -p * inner[m]
                err[m] = np.abs(p * inner[m]) * U32 * (2 * np.abs(np.where(p > 0, t, 0)) + E + 16) + p * e_inner[m]
    for m in range(M):
        for s in range(k):
            if live[m, s]:
                i = ids[m, s]
                out[m, i] += w[m, s] * (dw[m, s] - (inner[m, 0] if normalize else 0.0))
                err[m, i] += 4 * U32 * np.abs(w[m, s]) * (np.abs(dw[m, s]) + np.abs(inner[m, 0])) + \
                    (np.abs(w[m, s]) * e_inner[m, 0] if normalize else 0.0)
    return out, err + 4 * U32 * np.abs(out)


# ---------------------------------------------------------------------------
# the products: w is a list of each expert's W_hat [P][d]
# ---------------------------------------------------------------------------

def _expert_rows(offsets, order, k):
    for e in range(len(offsets) - 1):
        rows = np.arange(offsets[e], offsets[e + 1])
        if len(rows):
            yield e, rows, order[rows], order[rows] // k


def gated(offsets, order, k, x, w, bias, name):
    """(h [R][N], bound); rows behind the last pair: 0."""
    N = w[0].shape[0] // 2
    h, tol = np.zeros((len(order), N)), np.zeros((len(order), N))
    for e, rows, _, m in _expert_rows(offsets, order, k):
        b = None if bias is None else bias[e]
        h[rows] = block.gated(x[m], w[e], b, name)
        tol[rows] = block.gated_tolerance(x[m], w[e], b, name)
    return h, tol


def combine(offsets, order, k, h, w, bias, weights, residual):
    M = weights.shape[0]
    N = w[0].shape[0]
    y = np.zeros((M, N)) if residual is None else np.asarray(residual, np.float64).copy()
    size, err = np.abs(y), np.zeros((M, N))
    flat = np.asarray(weights, np.float64).reshape(-1)
    for e, rows, pairs, m in _expert_rows(offsets, order, k):
        z = block.preactivation(h[rows], w[e], None if bias is None else bias[e])
        share = flat[pairs][:, None]
        np.add.at(y, m, share * z)
        np.add.at(size, m, np.abs(share * z))
        np.add.at(err, m, np.abs(share) * (sum_error(h[rows], w[e]) + 2 * U32 * np.abs(z)))
    return y, rounded(y, err + (k + 2) * U32 * size)


def gated_backward_dz(offsets, order, k, x, w, bias, name, dh):
    P = w[0].shape[0]
    dz, tol = np.zeros((len(order), P)), np.zeros((len(order), P))
    for e, rows, _, m in _expert_rows(offsets, order, k):
        b = None if bias is None else bias[e]
        dz[rows] = block.gated_backward(x[m], w[e], b, name, dh[rows])[1]
        tol[rows] = block.grad_tolerance(x[m], w[e], b, name, dh[rows], True)
    return dz, tol


def gated_backward_dx(offsets, order, k, M, w, dz):
    """dx of the rounded dz that the device made."""
    d = w[0].shape[1]
    dx, err, size = np.zeros((M, d)), np.zeros((M, d)), np.zeros((M, d))
    for e, rows, _, m in _expert_rows(offsets, order, k):
        part = np.asarray(dz[rows], np.float64) @ w[e]
        np.add.at(dx, m, part)
        np.add.at(size, m, np.abs(part))
        np.add.at(err, m, sum_error(dz[rows], w[e].T.copy()))
    return dx, rounded(dx, err + (k + 2) * U32 * size)


def combine_backward(offsets, order, k, h, w, bias, weights, dy):
    """(dh, bound, dweights, bound)."""
    M, N = dy.shape
    d = w[0].shape[1]
    R = len(order)
    dh, dh_tol = np.zeros((R, d)), np.zeros((R, d))
    dw, dw_tol = np.zeros(R), np.zeros(R)
    flat = np.asarray(weights, np.float64).reshape(-1)
    for e, rows, pairs, m in _expert_rows(offsets, order, k):
        g, a = np.asarray(dy[m], np.float64), np.asarray(h[rows], np.float64)
        u, eu = g @ w[e], sum_error(dy[m], w[e].T.copy())
        share = flat[pairs][:, None]
        dh[rows] = share * u
        dh_tol[rows] = rounded(share * u, np.abs(share) * (eu + 2 * U32 * np.abs(u)))
        b = np.zeros(N) if bias is None else np.asarray(bias[e], np.float64)
        dw[pairs] = (u * a).sum(1) + g @ b
        dw_tol[pairs] = (np.abs(a) * eu).sum(1) + \
            (d + N + 4) * U32 * (np.abs(u * a).sum(1) + np.abs(g) @ np.abs(b))
    return dh, dh_tol, dw.reshape(M, k), dw_tol.reshape(M, k)


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def distill(z, values, index, lse, row_weight, T, scale, kind):
    """(loss [M], bound, dz [M][V], bound) for the student's type `kind`."""
    z = np.asarray(z, np.float64)
    M, V = z.shape
    loss, loss_tol = np.zeros(M), np.zeros(M)
    dz, dz_tol = np.zeros((M, V)), np.zeros((M, V))
    for m in range(M):
        w = 1.0 if row_weight is None else float(row_weight[m])
        at = (index[m] >= 0) & (index[m] < V)
        if w == 0.0 or (lse is None and not (at & ~(values[m] == -np.inf)).any()):
            continue
        t = np.asarray(values[m], np.float64)[at] / T
        j = index[m][at]
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            p_i = np.exp(t - t.max()) / np.exp(t - t.max()).sum() if lse is None else np.exp(t - float(lse[m]))
            P = 0.0 if lse is None else max(0.0, 1.0 - p_i.sum())
            A = 1.0 if lse is None else p_i.sum() + P
            target = np.zeros(V)
            np.add.at(target, j, p_i)
            entry = np.zeros(V, bool)
            entry[j] = True
            top = z[m].max()
            y = (z[m] - top) / T
            e = np.exp(y)
            total = e.sum()
            # the rest by itself, in the unit of its own largest: it may be far below the entries
            far = z[m][~entry].max() if lse is not None and not entry.all() else top
            own_y = (z[m] - far) / T if far > -np.inf else np.full(V, -np.inf)
            outside = np.where(entry, 0.0, np.exp(own_y)) if lse is not None else e
            left = outside.sum()
            own = np.where(p_i > 0, p_i * (np.log(p_i) - y[j]), np.where(p_i == 0, 0.0, np.nan)).sum()
            value = own + A * np.log(total)
            log_left = np.log(left) + (far - top) / T
            if P > 0:
                value += P * (np.log(P) - log_left)
            Q = left * np.exp((far - top) / T) / total
            r = outside / left if left > 0 else np.zeros(V)  # the student among the rest
            grad = np.where(entry, A * e / total, r * (A * Q - P) if lse is not None else A * e / total) - target
            # the fp32 sum of exponentials: arguments within 3 2^-24 of their size, a few ulps of exp2, at most
            # V / 256 + 16 additions and as many rescalings of a lane's sum, a tree over the lanes. (What is more
            # than 100 below the largest adds less than 2^20 e^-99 of the sum, whatever its argument's error.)
            span = min(np.abs(own_y[np.isfinite(own_y) & (outside > 0)]).max(initial=0.0), 100.0)
            sigma = U32 * (3 * span + 2 * (V / 256) + 80)
            rho = U32 * (3 * np.where(np.isfinite(own_y), np.abs(own_y), 0.0) + 8)
            share = Q if lse is not None else 1.0
            off = abs(Q * A - P) * sigma + P * sigma ** 2 if lse is not None else A * sigma
            loss[m] = w * T * T * value
            size = abs(own) + abs(np.log(total)) + abs(P * np.log(max(P, 1e-300))) + 1 + \
                (abs(P * log_left) if P > 0 else 0.0)
            loss_tol[m] = abs(w) * T * T * (off + 1e-13 * size)
            loss_tol[m] += U32 * (abs(loss[m]) + loss_tol[m]) + 2.0 ** -150
            g = w * T * scale
            dz[m] = g * grad
            if lse is None:
                err = np.abs(g) * (e / total) * np.where(entry, A * sigma, rho * A + A * sigma)
            else:
                err = np.abs(g) * np.where(entry, e / total * A * share * sigma,
                                           r * (rho * abs(A * Q - P) + sigma * (A * Q * Q + P)))
            err = err + 2 * U32 * np.abs(dz[m]) + 1e-14 * np.abs(g)
            dz_tol[m] = stored(dz[m], err, kind)
    return loss, loss_tol, dz, dz_tol
