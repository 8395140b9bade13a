"""The 16-bit expert FFN and its gradients in float64, expert by expert, each
with an elementwise error bound of the arithmetic the library documents:
float32 sums in any order, one nearest-even rounding per result, gradients of
the pre-activations rounded to the operands' type.

Bounds (u = 2^-24, h = half a step of the 16-bit type relative to the value,
tiny = half its smallest step):
  a sum of n products       n u sum|a b|
  exp, quotient, activation (16 + 2|g|) u relative (two ulp of exp, of the
                            quotient, and the rounded argument of exp)
  a result                  h |result| + tiny
The activations' first derivatives are below 1.13 and second ones below 1.2
in magnitude (SiLU: 1.1, 0.5; GELU: 1.13, 1.13)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
SLOPE, CURVE = 1.13, 1.2


def act(g, kind):
    """Activation and its derivative."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s + g * s * (1 - s)
    r = np.sqrt(2 / np.pi)
    t = np.tanh(r * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * r * (1 + 3 * 0.044715 * g * g)


def groups(offsets):
    for e in range(len(offsets) - 1):
        if offsets[e + 1] > offsets[e]:
            yield e, slice(int(offsets[e]), int(offsets[e + 1]))


def product(a, b, offsets, rows=None, dtype="bf16"):
    """y [offsets[-1], N] and its bound."""
    M = int(offsets[-1])
    y, tol = np.zeros((M, b.shape[1])), np.zeros((M, b.shape[1]))
    for e, s in groups(offsets):
        x = a[rows[s]] if rows is not None else a[s]
        y[s] = x @ b[e].T
        tol[s] = b.shape[2] * U * (np.abs(x) @ np.abs(b[e]).T)
    return y, tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(y) + TINY[dtype]


def _weight_grad(d, x, tol_d, n):
    return d.T @ x, tol_d.T @ np.abs(x) + n * U * ((np.abs(d) + tol_d).T @ np.abs(x))


def product_grad(dy, a, b, offsets, rows=None, dtype="bf16", tol_dy=None):
    """((da, bound), (db, bound)); tol_dy: bound of dy itself where it is a computed value."""
    M = int(offsets[-1])
    da, ta = np.zeros((M, b.shape[2])), np.zeros((M, b.shape[2]))
    db, tb = np.zeros(b.shape), np.zeros(b.shape)
    for e, s in groups(offsets):
        x = a[rows[s]] if rows is not None else a[s]
        d = dy[s]
        td = np.zeros_like(d) if tol_dy is None else tol_dy[s]
        da[s] = d @ b[e]
        ta[s] = td @ np.abs(b[e]) + b.shape[1] * U * ((np.abs(d) + td) @ np.abs(b[e]))
        db[e], tb[e] = _weight_grad(d, x, td, len(d))
    h, tiny = HALF[dtype], TINY[dtype]
    return (da, ta * (1 + h) + h * np.abs(da) + tiny), (db, tb * (1 + h) + h * np.abs(db) + tiny)


def gated(x, w, offsets, rows=None, kind="silu", dtype="bf16"):
    """((h, bound), (gu, bound))."""
    I = w.shape[1] // 2
    gu, tgu = product(x, w, offsets, rows, "f32")
    g, u, tg, tu = gu[:, :I], gu[:, I:], tgu[:, :I], tgu[:, I:]
    a, _ = act(g, kind)
    h = a * u
    tol = SLOPE * tg * (np.abs(u) + tu) + np.abs(a) * tu + (16 + 2 * np.abs(g)) * U * np.abs(h)
    return (h, tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(h) + TINY[dtype]), (gu, tgu)


def gated_grad(dh, x, w, offsets, rows=None, kind="silu", dtype="bf16"):
    """((dx, bound), (dw, bound)); dx one row per GEMM row."""
    I = w.shape[1] // 2
    gu, tgu = product(x, w, offsets, rows, "f32")
    M = len(gu)
    g, u, tg, tu = gu[:, :I], gu[:, I:], tgu[:, :I], tgu[:, I:]
    a, da = act(g, kind)
    d = np.abs(dh[:M])
    dgu = np.concatenate([dh[:M] * u * da, dh[:M] * a], 1)
    rel = (32 + 4 * np.abs(g)) * U
    # the slope is a sum of terms up to 1 + |g|: its float32 error is relative to those
    tol = np.concatenate([d * (CURVE * tg * (np.abs(u) + tu) + SLOPE * tu + rel * np.abs(u) * (1 + np.abs(g))),
                          d * (SLOPE * tg + rel * np.abs(a))], 1)
    tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dgu) + TINY[dtype]
    return product_grad(dgu, x, w, offsets, rows, dtype, tol)
