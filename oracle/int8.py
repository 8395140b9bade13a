"""INT8 with one scale per row: the quantiser (decisions in float32) and the
grouped product (exact integer sums)."""
from __future__ import annotations

import numpy as np

from .experts16 import HALF, TINY, U, act, groups


def quantize(x):
    """float32 x [..., cols] -> codes int8, scales float32."""
    x = np.asarray(x, np.float32)
    s = (np.abs(x).max(-1) * np.float32(1 / 127)).astype(np.float32)
    s = np.where(s > 0, s, np.float32(1))
    q = np.rint((x / s[..., None]).astype(np.float32))
    return np.clip(q, -127, 127).astype(np.int8), s


def grouped_gemm(a, sa, b, sb, offsets, rows=None):
    """y float64 [offsets[-1], N] from exact integer sums, and the bound of a
    float32 evaluation: the sum's conversion and two products, 3 roundings."""
    y = np.zeros((int(offsets[-1]), b.shape[1]))
    for e, s in groups(offsets):
        at = rows[s] if rows is not None else np.arange(s.start, s.stop)
        acc = a[at].astype(np.int64) @ b[e].astype(np.int64).T
        y[s] = acc * sa[at].astype(np.float64)[:, None] * sb[e].astype(np.float64)
    return y, 3.01 * U * np.abs(y)


def rounded(y, tol, dtype):
    """The bound after one more rounding to `dtype`."""
    return tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(y) + TINY[dtype]


def swiglu(y, tol):
    """h = silu(gate) * up of y [M, 2I] and the bound before its rounding."""
    I = y.shape[1] // 2
    g, u, tg, tu = y[:, :I], y[:, I:], tol[:, :I], tol[:, I:]
    a, _ = act(g, "silu")
    h = a * u
    return h, 1.13 * tg * (np.abs(u) + tu) + np.abs(a) * tu + (16 + 2 * np.abs(g)) * U * np.abs(h)
