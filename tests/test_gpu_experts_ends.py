"""The gated block at the ends of its activation: one row per expert with one
pre-activation g = u (exact), from -3e38 through the values where exp(-g)
overflows and s (1 - s) vanishes to 1e18.  h and every gradient against
float64, and zero where nothing contributes."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import experts16 as X
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu
G = [-3e38, -1e18, -1e4, -1000, -104, -90, -87, -60, -30, -18, -15, -12, -8, -6, -5, -4, -3, -1.28, -1, -1e-3, -1e-38, 0, 1e-38,
     1e-3, 1, 3, 4, 5, 6, 8, 12, 15, 18, 30, 60, 87, 90, 104, 1000, 1e4, 1e18]
U, HALF, TINY = X.U, X.HALF["bf16"], X.TINY["bf16"]


def _activation(g, kind):
    """a, its slope, and float32 bounds of both: the logistic s(z) to
    (16 + 8 |z|) U relative (argument, exp, sum, quotient) or 2^-126 where its exp
    overflows, the slope's terms to twice that each; exact beyond |g| = 200."""
    z = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        s, not_s = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    dz = np.ones_like(g) if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * g * g)
    near = np.abs(g) <= 200
    gn = np.where(near, np.abs(g), 0)
    rel = np.where(near, (16 + 8 * np.abs(z)) * U, 0)
    terms = s * (1 + gn * np.where(near, dz, 0))
    low = np.where(near, 2.0 ** -126, 0)
    slope = s + np.where(near, g * s * not_s * dz, 0)
    return g * s, slope, rel * s * gn + low * gn, 2 * rel * terms + low * (1 + gn * np.where(near, dz, 0)) + np.where(near, 4 * U * terms, 0)


@pytest.mark.parametrize("hint", [0, 5000, 200000])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ends_of_the_activation(kind, hint):
    print(f"ends {kind} hint {hint}", flush=True)
    I, H, E = 16, 8, len(G)
    x = torch.zeros((E, H), dtype=torch.bfloat16)
    x[:, 0] = torch.tensor(G, dtype=torch.float64).to(torch.bfloat16)
    g = x[:, 0].double().numpy()
    w = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16)
    w[:, :, 0] = 1
    w[:, :, 1] = 1                                # a second input column, 0 in x: dx has it too
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    kw = dict(activation=m.ACT_SILU if kind == "silu" else m.ACT_GELU, max_rows_per_expert_hint=hint)
    x, w = x.to(DEV), w.to(DEV)
    h, gu = m.moe_gated_ffn(x, w, off, m_total=E, save_gu=True, **kw)
    dh = torch.ones((E, I), dtype=torch.bfloat16, device=DEV)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off, **kw)
    assert np.array_equal(gu.double().cpu().numpy(), np.repeat(g[:, None], 2 * I, 1))
    a, slope, ta, ts = _activation(g, kind)

    def close(got, want, tol, what):
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all(), f"{what}: not finite"
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), f"{what} at g = {g[np.nonzero(bad)[0]]}: {got[bad]}, expected {np.broadcast_to(want, got.shape)[bad]}"

    def rounded(v, t):
        return t * (1 + HALF) + HALF * np.abs(v) + TINY

    want = a * g
    close(h, want[:, None], rounded(want, ta * np.abs(g) + U * np.abs(want))[:, None], "h")
    dg, du = g * slope, a                         # dh = 1
    tg, tu = rounded(dg, ts * np.abs(g) + U * np.abs(dg)), rounded(du, ta)
    want = I * (dg + du)                          # 2 I equal products: below 2 I float32 steps
    tol = rounded(want, I * (tg + tu) + 2 * I * U * I * (np.abs(dg) + tg + np.abs(du) + tu))
    close(dx[:, :2], want[:, None], tol[:, None], "dx")
    assert not dx[:, 2:].any()
    d = np.concatenate([np.repeat(dg[:, None], I, 1), np.repeat(du[:, None], I, 1)], 1)
    t = np.concatenate([np.repeat(tg[:, None], I, 1), np.repeat(tu[:, None], I, 1)], 1)
    want = d * g[:, None]
    close(dw[:, :, 0], want, rounded(want, t * np.abs(g[:, None]) + U * np.abs(want)), "dw")
    assert not dw[:, :, 1:].any()
    far = g < -200
    assert far.sum() == 4 and not h[torch.from_numpy(far)].any() and not dx[torch.from_numpy(far)].any()


@pytest.mark.parametrize("E", [300, 1025, 4096])
def test_gradients_of_many_experts(E):
    """Rows for a few of them: the activation's gradient past its task map's first 256 experts."""
    r = np.random.default_rng(E)
    counts = np.zeros(E, int)
    counts[[0, 3, 255, 256, 257, 270, E - 1]] = [4, 70, 1, 130, 64, 2, 65]
    off = np.concatenate([[0], np.cumsum(counts)])
    M, H, I, T = int(off[-1]), 40, 72, 50
    x = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w = torch.from_numpy((r.standard_normal((E, 2 * I, H)) * 0.2).astype(np.float32)).to(torch.bfloat16)
    dh = torch.from_numpy(r.standard_normal((M, I)).astype(np.float32)).to(torch.bfloat16)
    rows = r.integers(0, T, M).astype(np.int32)
    off_d, rows_d = torch.from_numpy(off.astype(np.int32)).to(DEV), torch.from_numpy(rows).to(DEV)
    xd, wd, dhd = x.to(DEV), w.to(DEV), dh.to(DEV)
    _, gu = m.moe_gated_ffn(xd, wd, off_d, m_total=M, a_rows=rows_d, save_gu=True)
    dx, dw = m.moe_gated_ffn_backward(dhd, gu, xd, wd, off_d, a_rows=rows_d)
    (rdx, tdx), (rdw, tdw) = X.gated_grad(dh.double().numpy(), x.double().numpy(), w.double().numpy(), off, rows)
    for got, want, tol in ((dx, rdx, tdx), (dw, rdw, tdw)):
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    assert not dw[torch.from_numpy(counts == 0).to(DEV)].any()
