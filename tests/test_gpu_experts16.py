"""The 16-bit expert FFN (moe_gated_ffn, moe_grouped_gemm) and its gradients
against float64 (oracle/experts16.py, whose bounds are derived there): types,
activations, group sizes from none to several tiles, odd sizes, gathered rows,
garbage where nothing may be read, untouched rows, streams and graphs."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import experts16 as X
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"silu": m.ACT_SILU, "gelu": m.ACT_GELU}


def _make(shape, dtype, r, std=1.0):
    """(GPU tensor, its exact float64 values)"""
    t = torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def _off(counts):
    off = np.concatenate([[0], np.cumsum(counts)])
    return off, torch.from_numpy(off.astype(np.int32)).to(DEV)


def _close(got, want, tol, what):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.nanmax(err / tol):.3f} of the bound"


# (rows of each expert, H, I): single tokens, empty experts, counts around the
# tile sizes, reductions below and across a step, sizes that are odd multiples of 8
GROUPS = [
    ([1], 64, 32), ([0, 1, 0, 2], 136, 40), ([8] * 5, 256, 128), ([17, 0, 63, 65], 264, 72), ([129, 5], 8, 8),
    ([0, 0, 300], 200, 136), ([257, 31, 1, 0, 16], 512, 256), ([15, 16, 17], 1032, 24),
    ([520], 320, 264), ([3, 700, 0, 64], 192, 128),
    # few rows an expert, short reductions, many tiles: the 64-row tiles (of both products)
    ([5] * 30 + [0, 70, 0, 129, 64] + [9] * 6, 136, 520), ([5] * 30 + [0, 70, 0, 129, 64] + [9] * 6, 1096, 136),
]
IDS = [f"{'-'.join(map(str, c)) if len(c) < 9 else f'{len(c)}experts'}x{h}x{i}" for c, h, i in GROUPS]


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu")])
@pytest.mark.parametrize("counts,H,I", GROUPS, ids=IDS)
def test_gated_block_and_gradients(counts, H, I, dtype, act):
    print(f"gated {counts} H={H} I={I} {dtype} {act}", flush=True)
    r = np.random.default_rng([H, I, len(counts)])
    off, off_d = _off(counts)
    M, E, T = int(off[-1]), len(counts), max(4, int(off[-1]) // 3)
    x, x64 = _make((T, H), dtype, r)
    w, w64 = _make((E, 2 * I, H), dtype, r, 1.5 / np.sqrt(H))
    dh, dh64 = _make((M, I), dtype, r)
    rows = r.integers(0, T, M).astype(np.int32)
    rows_d = torch.from_numpy(rows).to(DEV)
    kw = dict(a_rows=rows_d, activation=ACT[act])
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True, **kw)
    h2 = m.moe_gated_ffn(x, w, off_d, m_total=M, **kw)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, **kw)
    (rh, th), (rgu, tgu) = X.gated(x64, w64, off, rows, act, dtype)
    (rdx, tdx), (rdw, tdw) = X.gated_grad(dh64, x64, w64, off, rows, act, dtype)
    _close(h, rh, th, "h")
    assert torch.equal(h, h2)
    _close(gu, rgu, tgu, "gu")
    _close(dx, rdx, tdx, "dx")
    _close(dw, rdw, tdw, "dw")
    # the tile kernels, which the sizes alone would not choose here
    for hint in (5000, 200000):
        hh, gg = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True, max_rows_per_expert_hint=hint, **kw)
        _close(hh, rh, th, f"h, hint {hint}")
        _close(gg, rgu, tgu, f"gu, hint {hint}")
        ddx, ddw = m.moe_gated_ffn_backward(dh, gg, x, w, off_d, max_rows_per_expert_hint=hint, **kw)
        _close(ddx, rdx, tdx, f"dx, hint {hint}")
        _close(ddw, rdw, tdw, f"dw, hint {hint}")
    only_dx, none = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, need_dw=False, **kw)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, need_dx=False, **kw)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,K", GROUPS, ids=IDS)
def test_product_and_gradients(counts, N, K, dtype):
    print(f"product {counts} N={N} K={K} {dtype}", flush=True)
    r = np.random.default_rng([N, K, 7])
    off, off_d = _off(counts)
    M, E = int(off[-1]), len(counts)
    a, a64 = _make((M, K), dtype, r)
    b, b64 = _make((E, N, K), dtype, r, 1 / np.sqrt(K))
    dy, dy64 = _make((M, N), dtype, r)
    y = m.moe_grouped_gemm(a, b, off_d, m_total=M)
    y32 = m.moe_grouped_gemm(a, b, off_d, m_total=M, out_dtype=torch.float32)
    for hint in (5000, 200000):
        _close(m.moe_grouped_gemm(a, b, off_d, m_total=M, max_rows_per_expert_hint=hint), *X.product(a64, b64, off, None, dtype), "y")
        _close(m.moe_grouped_gemm(a, b, off_d, m_total=M, out_dtype=torch.float32, max_rows_per_expert_hint=hint),
               *X.product(a64, b64, off, None, "f32"), "y32")
        for got, (want, tol) in zip(m.moe_grouped_gemm_backward(dy, a, b, off_d, max_rows_per_expert_hint=hint),
                                    X.product_grad(dy64, a64, b64, off, None, dtype)):
            _close(got, want, tol, f"gradient, hint {hint}")
    da, db = m.moe_grouped_gemm_backward(dy, a, b, off_d)
    _close(y, *X.product(a64, b64, off, None, dtype), "y")
    _close(y32, *X.product(a64, b64, off, None, "f32"), "y32")
    (rda, tda), (rdb, tdb) = X.product_grad(dy64, a64, b64, off, None, dtype)
    _close(da, rda, tda, "da")
    _close(db, rdb, tdb, "db")
    rows = r.permutation(M).astype(np.int32)
    rows_d = torch.from_numpy(rows).to(DEV)
    y = m.moe_grouped_gemm(a, b, off_d, m_total=M, a_rows=rows_d)
    _, db = m.moe_grouped_gemm_backward(dy, a, b, off_d, a_rows=rows_d, need_da=False)
    _close(y, *X.product(a64, b64, off, rows, dtype), "gathered y")
    _close(db, *X.product_grad(dy64, a64, b64, off, rows, dtype)[1], "gathered db")


@pytest.mark.parametrize("hint", [1, 100, 5000, 100000])
def test_every_hint_gives_a_right_result(hint):
    r = np.random.default_rng(hint)
    counts, H, I = [40, 0, 300, 9], 328, 104
    off, off_d = _off(counts)
    M = int(off[-1])
    x, x64 = _make((M, H), "bf16", r)
    w, w64 = _make((4, 2 * I, H), "bf16", r, 0.1)
    dh, dh64 = _make((M, I), "bf16", r)
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True, max_rows_per_expert_hint=hint)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, max_rows_per_expert_hint=hint)
    _close(h, *X.gated(x64, w64, off)[0], "h")
    g1, g2 = X.gated_grad(dh64, x64, w64, off)
    _close(dx, *g1, "dx")
    _close(dw, *g2, "dw")


@pytest.mark.parametrize("hint", [4, 5000, 200000])
def test_garbage_outside_the_groups_is_neither_read_nor_written(hint):
    """NaN in unreferenced source rows, in rows behind the last expert and in the
    weights of empty experts stays there; result rows behind the last expert
    keep their bytes; an expert's NaN row stays in its own rows and its own
    weight gradient."""
    r = np.random.default_rng(5)
    counts, H, I, extra = [5, 0, 70, 33], 136, 72, 9
    off, off_d = _off(counts)
    M = int(off[-1]) + extra
    x, x64 = _make((M + 3, H), "bf16", r)
    w, w64 = _make((4, 2 * I, H), "bf16", r, 0.1)
    dh, dh64 = _make((M, I), "bf16", r)
    rows = np.concatenate([r.permutation(M + 3)[:off[-1]], np.full(extra, M + 2)]).astype(np.int32)
    unused = np.setdiff1d(np.arange(M + 3), rows[:off[-1]])
    x[torch.from_numpy(unused).to(DEV)] = float("nan")
    w[1] = float("nan")
    dh[off[-1]:] = float("nan")
    rows_d = torch.from_numpy(rows).to(DEV)
    out = torch.full((M, I), 7.0, dtype=torch.bfloat16, device=DEV)
    gu = torch.full((M, 2 * I), float("nan"), device=DEV)
    dx = torch.full((M, H), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(a_rows=rows_d, max_rows_per_expert_hint=hint)
    m.moe_gated_ffn(x, w, off_d, m_total=M, out=out, gu=gu, **kw)
    _, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, dx=dx, **kw)
    n = int(off[-1])
    (rh, th), _ = X.gated(x64, w64, off, rows)
    g1, g2 = X.gated_grad(dh64, x64, w64, off, rows)
    _close(out[:n], rh, th, "h")
    _close(dx[:n], *g1, "dx")
    _close(dw, *g2, "dw")
    assert (out[n:] == 7).all() and (dx[n:] == 7).all() and torch.isnan(gu[n:]).all()
    # one bad row: expert 2 only
    x[int(rows[20])] = float("inf")
    m.moe_gated_ffn(x, w, off_d, m_total=M, out=out, gu=gu, **kw)
    _, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, dx=dx, **kw)
    keep = [i for i in range(n) if i != 20]
    _close(out[keep], rh[keep], th[keep], "h beside a bad row")
    _close(dx[keep], g1[0][keep], g1[1][keep], "dx beside a bad row")
    for e in (0, 1, 3):
        _close(dw[e], g2[0][e], g2[1][e], f"dw[{e}]")
    assert not torch.isfinite(dw[2]).all()


# sizes that choose each kernel by themselves: many tiles of 128 x 128, many of
# 256 x 256 (with a last chunk of a few rows), and dense products whose row
# gradient is summed in parts
@pytest.mark.parametrize("counts,H,I", [([5] * 40, 1096, 520), ([300, 259, 256, 270, 512, 1, 330, 200], 2056, 1032),
                                        ([37], 136, 1160), ([130], 72, 2056)], ids=["tile128", "tile256", "parts", "parts2"])
def test_kernels_by_size(counts, H, I):
    r = np.random.default_rng([H, I])
    off, off_d = _off(counts)
    M, E = int(off[-1]), len(counts)
    x, x64 = _make((M, H), "bf16", r)
    w, w64 = _make((E, 2 * I, H), "bf16", r, 1 / np.sqrt(H))
    dh, dh64 = _make((M, I), "bf16", r)
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d)
    _close(h, *X.gated(x64, w64, off)[0], "h")
    g1, g2 = X.gated_grad(dh64, x64, w64, off)
    _close(dx, *g1, "dx")
    _close(dw, *g2, "dw")
    # two calls in one go on one workspace size, and again: the same bytes
    dx2, dw2 = m.moe_gated_ffn_backward(dh, gu, x, w, off_d)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    a, a64 = _make((M, I), "f16", r)
    b, b64 = _make((E, H, I), "f16", r, 1 / np.sqrt(I))
    dy, dy64 = _make((M, H), "f16", r)
    _close(m.moe_grouped_gemm(a, b, off_d, m_total=M), *X.product(a64, b64, off, None, "f16"), "y")
    da, db = m.moe_grouped_gemm_backward(dy, a, b, off_d)
    g1, g2 = X.product_grad(dy64, a64, b64, off, None, "f16")
    _close(da, *g1, "da")
    _close(db, *g2, "db")


def test_row_gradient_in_parts_leaves_rows_behind_the_last_expert():
    r = np.random.default_rng(31)
    off, off_d = _off([20, 0, 13])
    M, N, K = 40, 1024, 64
    need = m.lib().moe_grouped_gemm_backward_workspace_size(3, N, K, M)
    assert need > 0                       # the sizes do sum in parts
    a, a64 = _make((M, K), "bf16", r)
    b, b64 = _make((3, N, K), "bf16", r, 0.1)
    dy, dy64 = _make((M, N), "bf16", r)
    dy[33:] = float("nan")
    da = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)       # NaN patterns
    m.moe_grouped_gemm_backward(dy, a, b, off_d, da=da, need_db=False, workspace=ws)
    _close(da[:33], *X.product_grad(dy64, a64, b64, off)[0], "da")
    assert (da[33:] == 7).all()
    with pytest.raises(m.NVFP4MoEError):
        m.moe_grouped_gemm_backward(dy, a, b, off_d, workspace=ws[:need - 256])


@pytest.mark.parametrize("counts,H,I,parts", [([3000, 0, 5, 1501], 72, 40, 4), ([5003], 136, 200, 19),
                                              ([2700, 1, 900, 0, 260], 264, 136, 3), ([700, 1, 900, 0, 260], 264, 136, 0)],
                         ids=["small", "dense", "uneven", "one_part"])
def test_weight_gradient_in_parts_of_the_rows(counts, H, I, parts):
    """Few tiles and many rows: summed in parts, with the gathered and the direct rows, on a workspace of NaN."""
    r = np.random.default_rng([H, I, 5])
    off, off_d = _off(counts)
    M, E, T = int(off[-1]), len(counts), 911
    src = r.integers(0, T, M).astype(np.int32)
    x, x64 = _make((T, H), "bf16", r)
    w, w64 = _make((E, 2 * I, H), "bf16", r, 1 / np.sqrt(H))
    dh, dh64 = _make((M, I), "bf16", r)
    rows = torch.from_numpy(src).to(DEV)
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, a_rows=rows, save_gu=True)
    need = m.lib().moe_gated_ffn_backward_workspace_size(E, H, I, M)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, a_rows=rows, workspace=ws)
    g1, g2 = X.gated_grad(dh64, x64, w64, off, src)
    _close(dx, *g1, "dx")
    _close(dw, *g2, "dw")
    dy, dy64 = _make((M, 2 * I), "f16", r)
    a, a64 = _make((T, H), "f16", r)
    b, b64 = _make((E, 2 * I, H), "f16", r, 0.1)
    need = m.lib().moe_grouped_gemm_backward_workspace_size(E, 2 * I, H, M)
    assert need >= parts * E * 2 * I * H * 4
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    da, db = m.moe_grouped_gemm_backward(dy, a, b, off_d, a_rows=rows, workspace=ws)
    g1, g2 = X.product_grad(dy64, a64, b64, off, src, "f16")
    _close(da, *g1, "da")
    _close(db, *g2, "db")
    db2 = m.moe_grouped_gemm_backward(dy, a[rows.long()], b, off_d, need_da=False)[1]
    assert torch.equal(db, db2)


def test_row_gradient_of_a_badly_filled_last_round():
    """128 tiles of 256 x 256 on 256 CUs: summed in three parts of the reduction."""
    r = np.random.default_rng(12)
    M, N, K = 257, 6200, 16136
    assert m.lib().moe_grouped_gemm_backward_workspace_size(1, N, K, M + 7) == 3 * (M + 7) * K * 4
    _, off_d = _off([M])
    dy, dy64 = _make((M + 7, N), "bf16", r)
    b = torch.randn((1, N, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    da = torch.full((M + 7, K), 7.0, dtype=torch.bfloat16, device=DEV)
    m.moe_grouped_gemm_backward(dy, torch.empty((M + 7, K), dtype=torch.bfloat16, device=DEV), b.to(DEV), off_d, need_db=False, da=da)
    assert (da[M:] == 7).all()
    for k in range(0, K, 4096):
        b64 = b[0, :, k:k + 4096].double().numpy()
        want = dy64[:M] @ b64
        # at most N float32 additions in any order, then one rounding
        tol = N * X.U * (np.abs(dy64[:M]) @ np.abs(b64)) * (1 + X.HALF["bf16"]) + X.HALF["bf16"] * np.abs(want) + X.TINY["bf16"]
        _close(da[:M, k:k + 4096], want, tol, f"da from column {k}")


def test_activation_at_the_ends():
    """g far out on both sides: act(g) u without NaN, and its gradient."""
    g = torch.tensor([-3e38, -1e4, -100, -20, -1, 0, 1, 20, 100, 1e4], dtype=torch.float32)
    I, H = 16, 8
    w = torch.zeros((1, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    w[0, :, 0] = 1
    x = torch.zeros((len(g), H), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = g.to(torch.bfloat16).to(DEV)
    off = torch.tensor([0, len(g)], dtype=torch.int32, device=DEV)
    x64 = x.double().cpu().numpy()
    for kind in ("silu", "gelu"):
        h, gu = m.moe_gated_ffn(x, w, off, m_total=len(g), activation=ACT[kind], save_gu=True)
        dh = torch.ones((len(g), I), dtype=torch.bfloat16, device=DEV)
        dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off, activation=ACT[kind])
        ok = slice(1, None)           # -3e38 squared or cubed leaves float32: only its value is checked
        with np.errstate(over="ignore"):
            (rh, th), _ = X.gated(x64[ok], w.double().cpu().numpy(), np.array([0, len(g) - 1]), None, kind)
        _close(h[ok], rh, th, f"{kind} h")
        assert torch.isfinite(dx[2:].float()).all()


@pytest.mark.parametrize("E", [1, 3])
def test_no_rows_at_all(E):
    H, I = 64, 32
    w = torch.randn((E, 2 * I, H), device=DEV).to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    x = torch.empty((0, H), dtype=torch.bfloat16, device=DEV)
    h, gu = m.moe_gated_ffn(x, w, off, m_total=0, save_gu=True)
    assert h.shape == (0, I) and gu.shape == (0, 2 * I)
    dx, dw = m.moe_gated_ffn_backward(h, gu, x, w, off)
    assert dx.shape == (0, H) and not dw.any()
    assert m.moe_grouped_gemm(x, w, off, m_total=0).shape == (0, 2 * I)
    da, db = m.moe_grouped_gemm_backward(torch.empty((0, 2 * I), dtype=torch.bfloat16, device=DEV), x, w, off)
    assert da.shape == (0, H) and not db.any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert m.moe_gated_ffn(x, w, off, m_total=0, stream=side).shape == (0, I)
    dx, dw = m.moe_gated_ffn_backward(h, gu, x, w, off, stream=side)
    side.synchronize()
    assert dx.shape == (0, H) and not dw.any()


def test_more_experts_than_one_scan_group():
    """300 experts, most of them empty: the task map's second group of 256."""
    r = np.random.default_rng(8)
    counts = np.zeros(300, int)
    counts[[0, 3, 255, 256, 270, 299]] = [4, 70, 1, 130, 2, 3]
    off, off_d = _off(counts)
    M = int(off[-1])
    a, a64 = _make((M, 72), "bf16", r)
    b, b64 = _make((300, 80, 72), "bf16", r, 0.1)
    dy, dy64 = _make((M, 80), "bf16", r)
    _close(m.moe_grouped_gemm(a, b, off_d, m_total=M), *X.product(a64, b64, off), "y")
    da, db = m.moe_grouped_gemm_backward(dy, a, b, off_d)
    g1, g2 = X.product_grad(dy64, a64, b64, off)
    _close(da, *g1, "da")
    _close(db, *g2, "db")


@pytest.mark.parametrize("E", [1023, 1024, 1025, 4096])
def test_many_experts(E):
    """Up to the limit, rows for about half of them: the map of 64-row tiles ends at 1024."""
    r = np.random.default_rng(E)
    counts = r.integers(0, 3, E) * r.integers(0, 2, E)
    counts[[0, E // 2, E - 1]] = [70, 130, 65]
    off, off_d = _off(counts)
    M = int(off[-1])
    a, a64 = _make((M, 40), "f16", r)
    b, b64 = _make((E, 24, 40), "f16", r, 0.2)
    _close(m.moe_grouped_gemm(a, b, off_d, m_total=M), *X.product(a64, b64, off, None, "f16"), "y")
    w, w64 = _make((E, 16, 40), "f16", r, 0.2)
    _close(m.moe_gated_ffn(a, w, off_d, m_total=M), *X.gated(a64, w64, off, None, "silu", "f16")[0], "h")


def test_gradients_against_differences_on_the_gpu():
    """The float32 loss sum(h * c) moved along one direction of x and of w:
    (loss(+) - loss(-)) / 2 eps from float64 forms against the GPU's gradients
    contracted with that direction; their bound is the elementwise one."""
    r = np.random.default_rng(11)
    counts, H, I = [20, 0, 45], 96, 40
    off, off_d = _off(counts)
    M = int(off[-1])
    x, x64 = _make((M, H), "bf16", r)
    w, w64 = _make((3, 2 * I, H), "bf16", r, 0.15)
    c, c64 = _make((M, I), "bf16", r)
    _, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True)
    dx, dw = m.moe_gated_ffn_backward(c, gu, x, w, off_d)
    (_, tdx), (_, tdw) = X.gated_grad(c64, x64, w64, off)
    vx, vw = r.standard_normal(x64.shape), r.standard_normal(w64.shape)
    eps = 1e-5

    def loss(a, b):
        return float((X.gated(a, b, off)[0][0] * c64).sum())

    num = (loss(x64 + eps * vx, w64) - loss(x64 - eps * vx, w64)) / (2 * eps)
    assert abs(num - float((dx.double().cpu().numpy() * vx).sum())) <= (tdx * np.abs(vx)).sum() + 1e-4
    num = (loss(x64, w64 + eps * vw) - loss(x64, w64 - eps * vw)) / (2 * eps)
    assert abs(num - float((dw.double().cpu().numpy() * vw).sum())) <= (tdw * np.abs(vw)).sum() + 1e-4


def test_side_stream_and_replayed_graph():
    """A step of forward and backward on another stream, then captured and
    replayed with new contents between eager runs: the same bytes."""
    r = np.random.default_rng(12)
    counts, H, I = [64, 3, 200], 256, 128
    off, off_d = _off(counts)
    M = int(off[-1])
    x, _ = _make((M, H), "bf16", r)
    w, _ = _make((3, 2 * I, H), "bf16", r, 0.1)
    dh, _ = _make((M, I), "bf16", r)

    def bufs():
        e = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device=DEV)   # noqa: E731
        n = m.lib().moe_gated_ffn_backward_workspace_size(3, H, I, M)
        return dict(out=e(M, I), gu=e(M, 2 * I, d=torch.float32)), dict(dx=e(M, H), dw=e(3, 2 * I, H), workspace=e(n, d=torch.uint8))

    def step(f, b, stream=None):
        m.moe_gated_ffn(x, w, off_d, m_total=M, stream=stream, **f)
        m.moe_gated_ffn_backward(dh, f["gu"], x, w, off_d, stream=stream, **b)

    f0, b0 = bufs()
    f1, b1 = bufs()
    step(f0, b0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(f1, b1, side)
    torch.cuda.synchronize()
    for k in ("out", "gu"):
        assert torch.equal(f0[k], f1[k])
    for k in ("dx", "dw"):
        assert torch.equal(b0[k], b1[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(f1, b1)
    for i in range(4):
        x.copy_(_make((M, H), "bf16", r)[0])
        dh.copy_(_make((M, I), "bf16", r)[0])
        for t in (f1["out"], f1["gu"], b1["dx"], b1["dw"]):
            t.zero_()
        graph.replay()
        step(f0, b0)
        torch.cuda.synchronize()
        assert torch.equal(f0["out"], f1["out"]) and torch.equal(b0["dx"], b1["dx"]) and torch.equal(b0["dw"], b1["dw"]), i


@pytest.mark.parametrize("hint", [0, 5000, 200000])
def test_bad_gather_entries_read_row_0(hint):
    """The kernels' own bound on the index array, in every product that gathers."""
    r = np.random.default_rng(41)
    off, off_d = _off([30, 50])
    x, _ = _make((20, 136), "bf16", r)
    w, _ = _make((2, 208, 136), "bf16", r, 0.1)
    dh, _ = _make((80, 104), "bf16", r)
    rows = r.integers(0, 20, 80).astype(np.int32)
    good = rows.copy()
    rows[[3, 31, 79]], good[[3, 31, 79]] = [-1, 20, 2 ** 31 - 1], 0
    res = []
    for q in (rows, good):
        kw = dict(a_rows=torch.from_numpy(q).to(DEV), max_rows_per_expert_hint=hint)
        h, gu = m.moe_gated_ffn(x, w, off_d, m_total=80, save_gu=True, **kw)
        dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d, need_dx=False, **kw)[1]
        dy = torch.cat([dh, dh], 1).contiguous()
        db = m.moe_grouped_gemm_backward(dy, x, w, off_d, need_da=False, **kw)[1]
        res.append((h, gu, dw, m.moe_grouped_gemm(x, w, off_d, m_total=80, **kw), db))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_debug_checks_cover_the_new_calls(monkeypatch):
    """With NVFP4MOE_DEBUG bad index arrays are refused on the host, before any launch."""
    monkeypatch.setenv("NVFP4MOE_DEBUG", "1")
    x = torch.zeros((20, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device=DEV)
    gu, dh = torch.zeros((20, 64), device=DEV), torch.zeros((20, 32), dtype=torch.bfloat16, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    rows = i32(*([0] * 19 + [20]))
    q = m.int8_quantize(x)
    wq = m.int8_quantize(w)
    for off, kw, text in ((i32(0, 12, 5), {}, "offsets decrease"), (i32(0, 12, 21), {}, "m_total"),
                          (i32(0, 12, 20), dict(a_rows=rows), "a_rows[19] = 20")):
        for call in (lambda: m.moe_gated_ffn(x, w, off, m_total=20, **kw),
                     lambda: m.moe_gated_ffn_backward(dh, gu, x, w, off, **kw),
                     lambda: m.moe_grouped_gemm(x, w, off, m_total=20, **kw),
                     lambda: m.moe_grouped_gemm_backward(x, x, w, off, **kw),
                     lambda: m.int8_grouped_gemm(q, wq, off, m_total=20, **kw)):
            with pytest.raises(m.NVFP4MoEError) as e:
                call()
            assert e.value.status == m.ERR_INVALID and text in e.value.detail


def test_backward_on_another_stream_with_its_own_workspace():
    """The call's temporary workspace is not handed out again while the stream
    it works on has not finished."""
    r = np.random.default_rng(43)
    off, off_d = _off([400, 300])
    x, _ = _make((700, 512), "bf16", r)
    w, _ = _make((2, 1024, 512), "bf16", r, 0.05)
    dh, _ = _make((700, 512), "bf16", r)
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=700, save_gu=True)
    want = m.moe_gated_ffn_backward(dh, gu, x, w, off_d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn((2048, 2048), device=DEV)
    n = m.lib().moe_gated_ffn_backward_workspace_size(2, 512, 512, 700)
    for _ in range(4):
        dx, dw = torch.empty_like(want[0]), torch.empty_like(want[1])
        with torch.cuda.stream(side):
            busy @ busy
        m.moe_gated_ffn_backward(dh, gu, x, w, off_d, dx=dx, dw=dw, stream=side)
        torch.full((n,), 255, dtype=torch.uint8, device=DEV)          # would take the freed block
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_two_streams_at_once():
    """Calls of different sizes side by side on two streams give what they give one after another."""
    r = np.random.default_rng(44)
    sets = []
    for counts, H, I in (([300, 20, 129], 512, 1032), ([7] * 60, 264, 520)):
        off, off_d = _off(counts)
        x, _ = _make((int(off[-1]), H), "bf16", r)
        w, _ = _make((len(counts), 2 * I, H), "bf16", r, 0.05)
        dh, _ = _make((int(off[-1]), I), "bf16", r)
        sets.append((x, w, dh, off_d, int(off[-1])))

    def both(x, w, dh, off_d, M, stream=None):
        h, gu = m.moe_gated_ffn(x, w, off_d, m_total=M, save_gu=True, stream=stream)
        return (h, gu) + m.moe_gated_ffn_backward(dh, gu, x, w, off_d, stream=stream)

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [both(*s, stream=q) for s, q in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_wrong_operands_are_refused():
    H, I = 64, 32
    x = torch.zeros((4, H), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    f = m.moe_gated_ffn
    with pytest.raises(TypeError):
        f(x.float(), w, off, m_total=4)
    with pytest.raises(TypeError):
        f(x.half(), w, off, m_total=4)
    with pytest.raises(ValueError):
        f(x[:, :32], w, off, m_total=4)
    with pytest.raises(ValueError):
        f(x.t().contiguous().t(), w, off, m_total=4)
    with pytest.raises(ValueError):
        f(x, w, off, m_total=5)
    with pytest.raises(ValueError):
        f(x, w, off[:2].contiguous(), m_total=4)
    with pytest.raises(ValueError):
        f(x.cpu(), w, off, m_total=4)
    with pytest.raises(ValueError):
        f(x, w, off, m_total=4, out=torch.empty((4, I + 8), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(m.NVFP4MoEError):
        f(x, w, off, m_total=4, activation=9)
    with pytest.raises(m.NVFP4MoEError):
        f(x[:, :12].contiguous(), w[:, :, :12].contiguous(), off, m_total=4)
    h, gu = f(x, w, off, m_total=4, save_gu=True)
    with pytest.raises(TypeError):
        m.moe_gated_ffn_backward(h.float(), gu, x, w, off)
    with pytest.raises(ValueError):
        m.moe_gated_ffn_backward(h, gu[:, :I].contiguous(), x, w, off)
    with pytest.raises(ValueError):
        m.moe_gated_ffn_backward(h, gu, x, w, off, need_dx=False, need_dw=False)
    with pytest.raises(m.NVFP4MoEError):
        m.moe_gated_ffn_backward(h, gu, x, w, off, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        m.moe_grouped_gemm(x, w, off, m_total=4, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        m.moe_grouped_gemm_backward(h, x, w, off)
