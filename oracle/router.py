"""The router with scores and the gradients of its logits and of the weighted
combine, token by token in float64, with elementwise bounds of the arithmetic the
library documents (u = 2^-24, HALF and TINY as in experts16)."""
from __future__ import annotations

import numpy as np

from .experts16 import HALF, TINY, U

F32_MAX = float(np.finfo(np.float32).max)


def scores(logits, kind):
    """Scores float64 [T, E] and which experts are open by their logit."""
    l = np.asarray(logits, np.float64)
    is_open = l > -np.inf                                  # neither -inf nor NaN
    x = np.minimum(np.where(is_open, l, 0.0), F32_MAX)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(is_open, 1 / (1 + np.exp(-x)), 0.0), is_open
    s = np.zeros(l.shape)
    for t in range(l.shape[0]):
        o = is_open[t]
        if o.any():
            e = np.exp(x[t, o] - x[t, o].max())
            s[t, o] = e / e.sum()
    return s, is_open


def weights(logits, ids, is_open, kind, renormalize, scale):
    """Weights [T, k] of chosen ids, float64; is_open [T, E]."""
    T, k = ids.shape
    at = np.arange(T)[:, None]
    x = np.minimum(np.where(is_open, np.asarray(logits, np.float64), 0.0), F32_MAX)[at, ids]
    o = is_open[at, ids]
    if not renormalize:
        return np.where(o, scores(logits, kind)[0][at, ids], 0.0) * scale
    w = np.zeros((T, k))
    for t in range(T):
        if not o[t].any():
            continue
        xt = x[t, o[t]]
        if kind == "softmax":
            u = np.exp(xt - xt.max())
        else:                                              # sigmoid * exp(-b): b divides out
            b = min(xt.max(), 0.0)
            with np.errstate(over="ignore"):
                u = 1 / (np.exp(b) + np.exp(b - xt))
        w[t, o[t]] = u / u.sum()
    return w * scale


def route(logits, k, kind="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k], scores float64 [T, E], open [T, E])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s, is_open = scores(l, kind)
    with np.errstate(invalid="ignore"):
        key = s + (0 if bias is None else np.asarray(bias, np.float64)[None, :])
    is_open = is_open & (key > -np.inf)
    order = key if bias is not None else np.minimum(l, F32_MAX)
    size = E // n_group
    ids = np.empty((T, k), np.int32)
    for t in range(T):
        values = []
        for g in range(n_group):
            keys = sorted((key[t, e] for e in range(g * size, (g + 1) * size) if is_open[t, e]), reverse=True)
            values.append(sum(keys[:group_top]) if keys else -np.inf)
        kept = set(sorted(range(n_group), key=lambda g: (-values[g], g))[:topk_group])
        allowed = [e for e in range(E) if e // size in kept]
        best = sorted((e for e in allowed if is_open[t, e]), key=lambda e: (-order[t, e], e))
        rest = [e for e in allowed if not is_open[t, e]]
        ids[t] = (best + rest)[:k]
    return ids, weights(l, ids, is_open, kind, renormalize, scale), s, is_open


def route_grad(dw, logits, ids, is_open, kind, renormalize, scale, d_scores=None, dtype="f32"):
    """Gradient of the logits and its bound for float32 arithmetic: relative errors
    of a softmax (|x - max| + E + 8) u, of a sigmoid (|x| + 8) u, of normalised weights
    the largest of those over the chosen plus (k + 8) u; sums of n terms n u of
    their magnitudes; one rounding to dtype."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = ids.shape[1]
    s, by_logit = scores(l, kind)
    x = np.minimum(np.where(by_logit, l, 0.0), F32_MAX)
    q = np.zeros((T, E)) if d_scores is None else np.broadcast_to(np.asarray(d_scores, np.float64), (T, E))
    out, tol = np.zeros((T, E)), np.zeros((T, E))
    wn = weights(l, np.clip(ids, 0, E - 1), is_open, kind, renormalize, 1.0)
    for t in range(T):
        o = by_logit[t]
        if not o.any():
            continue
        span = np.abs(x[t] - (x[t, o].max() if kind == "softmax" else 0.0))
        rs = (np.where(o, span, 0) + (E if kind == "softmax" else 0) + 8) * U
        inside = (ids[t] >= 0) & (ids[t] < E)
        chosen = np.clip(ids[t], 0, E - 1)
        n = np.where(inside, wn[t], 0.0)
        g = np.where(n > 0, np.asarray(dw[t], np.float64), 0.0)
        if renormalize:
            if not inside.all():                           # the share of those that count
                n = n / n.sum() if n.sum() > 0 else n
            alive = is_open[t, chosen] & inside
            far = np.abs(x[t, chosen] - x[t, chosen][alive].max())[alive].max() if alive.any() else 0.0
            if kind == "sigmoid" and alive.any():
                far += np.abs(x[t, chosen][alive]).max()
            rn = (far + k + 8) * U
            c = scale * n * (g - (g * n).sum())
            ec = abs(scale) * n * (np.abs(g) + (np.abs(g) * n).sum()) * (2 * rn + (k + 8) * U)
        else:
            c = scale * n * g
            ec = np.abs(c) * (rs[chosen] + 4 * U)
        ce, ece, mag = np.zeros(E), np.zeros(E), np.zeros(E)
        np.add.at(ce, chosen[inside], c[inside])
        np.add.at(ece, chosen[inside], ec[inside] + 2 * U * k * np.abs(c[inside]))
        np.add.at(mag, chosen[inside], np.abs(c[inside]))
        if kind == "sigmoid":
            with np.errstate(over="ignore"):
                rest = np.where(o, 1 / (1 + np.exp(x[t])), 0.0)
            out[t] = rest * (ce + s[t] * q[t])
            tol[t] = rest * (ece + (mag + s[t] * np.abs(q[t])) * (2 * rs + 8 * U))
        else:
            total = 0.0 if renormalize else c[inside].sum()
            qs, aq = (s[t] * q[t]).sum(), (s[t] * np.abs(q[t])).sum()
            out[t] = ce + s[t] * (q[t] - qs - total)
            spread = np.abs(q[t]) + aq + (0.0 if renormalize else mag.sum())
            tol[t] = ece + s[t] * (spread * (rs + rs.max() + (E + k + 8) * U) + (0.0 if renormalize else ece.sum())) + 4 * U * mag
        out[t, ~o], tol[t, ~o] = 0.0, 0.0
    return out, tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(out) + TINY[dtype] + 2.0 ** -125


def combine_grad(dout, y, rows, w, dtype="bf16"):
    """((dy, bound), (dw, bound)) of out[t] = sum_j w[t, j] y[rows[t, j]]: one float32
    product and a rounding; a float32 sum of H products."""
    T, k = rows.shape
    dy, dw = np.zeros(y.shape), np.zeros((T, k))
    tw = np.zeros((T, k))
    for j in range(k):
        dy[rows[:, j]] = w[:, j:j + 1].astype(np.float64) * dout
        dw[:, j] = (dout * y[rows[:, j]]).sum(1)
        tw[:, j] = y.shape[1] * U * np.abs(dout * y[rows[:, j]]).sum(1)
    return (dy, np.abs(dy) * (U + HALF[dtype] * (1 + U)) + TINY[dtype]), (dw, tw + U * np.abs(dw) + TINY["f32"])
