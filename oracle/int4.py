"""INT4 in groups along the last axis: the quantiser (decisions in float32), the
values of its codes, and the grouped product in float64 with a bound of the
library's arithmetic."""
from __future__ import annotations

import numpy as np

from .experts16 import HALF, SLOPE, TINY, U, act, groups


def round16(x, dtype):
    """float32 -> the nearest bf16 or f16 value (ties to even, overflow to infinity), as float32."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float16).float().numpy()


def quantize(x, group, zeros, dtype):
    """float32 x [..., cols] -> codes uint8 [..., cols/2], scales float32 (16-bit
    values) and zero points [..., cols/group] (None without)."""
    x = np.asarray(x, np.float32)
    v = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(invalid="ignore", over="ignore"):
        if zeros:
            lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
            s = ((hi - lo).astype(np.float32) * np.float32(1 / 15)).astype(np.float32)
        else:
            s = (np.abs(v).max(-1) * np.float32(1 / 7)).astype(np.float32)
        s = round16(s, dtype)
    good = np.isfinite(s) & np.isfinite(v).all(-1)
    s = np.where(good, np.where(s == 0, np.float32(1), s), np.float32(1)).astype(np.float32)
    v = np.where(good[..., None], v, 0).astype(np.float32)
    z = np.full(s.shape, 8.0)
    if zeros:
        z = np.clip(np.rint((-np.where(good, lo, 0).astype(np.float32) / s).astype(np.float32)), 0, 15)
    q = np.clip(np.rint((v / s[..., None]).astype(np.float32)) + z[..., None], 0, 15)
    q = np.where(good[..., None], q, 0 if zeros else 8).astype(np.uint8).reshape(x.shape)
    scales = np.where(good, s, np.float32(np.nan)).astype(np.float32)
    return q[..., 0::2] | (q[..., 1::2] << 4), scales, (np.where(good, z, 0).astype(np.uint8) if zeros else None)


def integers(codes, zeros, group):
    """code - zero, float64 [..., cols]."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, -1)
    return q - z


def dequantize(codes, scales, zeros, group):
    return integers(codes, zeros, group) * np.repeat(scales.astype(np.float64), group, -1)


def grouped(x, codes, scales, zeros, group, offsets, rows=None):
    """y float64 [offsets[-1], N] and its bound.  A group's sum runs over products
    with 16 + q and over the offset 16 + z that comes off (together below 64 |x| for
    each value, 2 group + 4 additions in float32, an error of 2 u each allowed for
    the matrix instruction's); scaled sums of K / group groups and up to 8 waves."""
    M, E, N = int(offsets[-1]), codes.shape[0], codes.shape[1]
    y, tol = np.zeros((M, N)), np.zeros((M, N))
    for e, at in groups(offsets):
        xe = (x[at] if rows is None else x[rows[at]]).astype(np.float64)
        b = dequantize(codes[e], scales[e], None if zeros is None else zeros[e], group)
        y[at] = xe @ b.T
        big = np.abs(xe).reshape(xe.shape[0], -1, group).sum(-1) @ np.abs(scales[e].astype(np.float64)).T
        tol[at] = 2 * U * (2 * group + 4) * 64 * big + (x.shape[1] / group + 16) * U * (np.abs(xe) @ np.abs(b).T + 64 * U * big)
    return y, tol


def rounded(y, tol, dtype):
    return tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(y) + TINY[dtype]


def gated(y, tol, kind):
    """h = act(gate) * up of y [M, 2I] and the bound before its rounding."""
    I = y.shape[1] // 2
    g, u, tg, tu = y[:, :I], y[:, I:], tol[:, :I], tol[:, I:]
    a, _ = act(g, kind)
    h = a * u
    return h, SLOPE * tg * (np.abs(u) + tu) + np.abs(a) * tu + (16 + 2 * np.abs(g)) * U * np.abs(h)
