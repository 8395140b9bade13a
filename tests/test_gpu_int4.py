"""INT4 quantiser, its inverse and products of few rows against oracle/int4.py:
codes, scales and zero points bit for bit, products within the bound of float32
sums."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import int4 as Q
from oracle.experts16 import HALF, TINY
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu

F = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"silu": m.ACT_SILU, "gelu": m.ACT_GELU}


def _bits(t):
    return t.cpu().view(torch.int16).numpy()


def _same_scales(got, want, st):
    """Bit for bit, a NaN being a NaN."""
    w = torch.from_numpy(want).to(F[st])
    g = got.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    ok = ~torch.isnan(w)
    assert torch.equal(g[ok].view(torch.int16), w[ok].view(torch.int16))


@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("st", ["bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (3, 96, 32), (37, 6144, 128), (5, 320, 64), (130, 128, 128), (1, 8192, 64)])
def test_quantize_bits(rows, cols, group, dtype, st, zeros):
    print("int4 quantize", rows, cols, group, dtype, st, zeros, flush=True)
    r = np.random.default_rng([rows, cols, group])
    x = (r.standard_normal((rows, cols)) * 10.0 ** r.integers(-4, 3, (rows, 1))).astype(np.float32)
    if rows > 1:
        x[1] = 0                                            # scale 1
    if rows > 2 and cols > group:
        x[2, :group] = np.where(np.arange(group) % 2, 1e-40, -1e-42)     # scales that round to 0, or hold few bits
        x[2, group:2 * group] = 3e-7
    if rows > 4:
        x[3, 0], x[3, min(group + 5, cols - 1)], x[4, -1] = np.nan, np.inf, -np.inf
    if rows > 4 and cols > 2 * group:
        x[4, :group] = np.abs(x[4, :group]) + 1             # one sign: the zero point at its end
        x[4, group:2 * group] = -x[4, :group]
        k = np.arange(group) % 16 - 8                       # every code and the ties between them
        x[3, 2 * group:3 * group] = (k + 0.5 * (np.arange(group) >= 16)) * 0.125
    t = torch.from_numpy(x).to(F[dtype])
    q = m.int4_quantize(t.to(DEV), group, zeros, F[st])
    codes, s, z = Q.quantize(t.float().numpy(), group, zeros, st)
    _same_scales(q.scales, s, st)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert (q.zeros is None) == (not zeros) and (not zeros or np.array_equal(q.zeros.cpu().numpy(), z))
    # and back: exact in float32, one rounding in 16 bits
    v = Q.dequantize(codes, s, z, group)
    got = m.int4_dequantize(q, torch.float32).cpu().numpy()
    assert np.array_equal(got[~np.isnan(v)].astype(np.float64), v[~np.isnan(v)]) and np.array_equal(np.isnan(got), np.isnan(v))
    got16 = m.int4_dequantize(q)
    want16 = torch.from_numpy(v.astype(np.float32)).to(F[st])
    ok = ~torch.isnan(want16)
    assert got16.dtype == F[st] and torch.equal(got16.cpu()[ok], want16[ok])


def test_quantize_dense_quotients():
    """Quotients k + 1/2 moved by a few float32 steps, for many scales: the division has to be the correctly rounded one."""
    r = np.random.default_rng(6)
    rows, group = 4096, 128
    top = (2.0 ** r.uniform(-20, 20, rows)).astype(np.float32)
    s = Q.round16((top * np.float32(1 / 7)).astype(np.float32), "bf16")
    k = r.integers(-6, 6, (rows, group)) + 0.5
    x = (k * s[:, None].astype(np.float64)).astype(np.float32)
    x = (x.view(np.int32) + r.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    x[:, 0] = top
    for zeros in (False, True):
        q = m.int4_quantize(up(x), group, zeros)
        codes, sc, z = Q.quantize(x, group, zeros, "bf16")
        _same_scales(q.scales, sc, "bf16")
        assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_quantize_shapes():
    x = torch.randn((2, 3, 5, 64), device=DEV)
    q = m.int4_quantize(x, 32)
    assert q.codes.shape == (2, 3, 5, 32) and q.scales.shape == (2, 3, 5, 2) and q.scales.dtype == torch.bfloat16
    again = m.int4_quantize(x, 32, out=m.INT4Tensor(torch.empty_like(q.codes), torch.empty_like(q.scales), None, 32))
    assert torch.equal(again.codes, q.codes) and torch.equal(_t16(again.scales), _t16(q.scales))
    assert m.int4_quantize(x[:0], 32).codes.shape == (0, 3, 5, 32) and m.int4_dequantize(m.int4_quantize(x[:0], 32)).numel() == 0


def _t16(t):
    return t.view(torch.int16)


# counts of rows per expert, N, K, group
SHAPES = [
    ([1], 1, 32, 32), ([1], 17, 128, 128), ([0, 1, 0, 2], 48, 192, 64), ([3], 63, 4096, 128), ([16], 40, 640, 64),
    ([17, 0, 63, 65], 66, 352, 32), ([5, 16, 1], 250, 256, 128), ([129, 5], 34, 576, 64), ([8] * 20, 130, 256, 64),
    ([2] * 40 + [0, 31], 96, 1152, 128), ([1, 33], 520, 2080, 32), ([300], 26, 96, 32), ([7, 9], 1030, 64, 64),
    ([1, 1, 0, 1], 256, 6144, 128), ([40] * 3, 256, 1024, 128),
]


@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,K,group", SHAPES, ids=[f"{'-'.join(map(str, c)) if len(c) < 6 else f'{len(c)}experts'}x{n}x{k}g{g}" for c, n, k, g in SHAPES])
def test_grouped_product(counts, N, K, group, dtype, zeros):
    print("int4 product", counts, N, K, group, dtype, zeros, flush=True)
    r = np.random.default_rng([N, K, group])
    off = np.concatenate([[0], np.cumsum(counts)])
    M, E, T = int(off[-1]), len(counts), 40
    codes = r.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    s = torch.from_numpy((r.standard_normal((E, N, K // group)) * 0.02).astype(np.float32)).to(F[dtype])
    z = r.integers(0, 16, (E, N, K // group)).astype(np.uint8) if zeros else None
    x = torch.from_numpy((r.standard_normal((T, K)) + 0.5).astype(np.float32)).to(F[dtype])
    rows = r.integers(0, T, M).astype(np.int32)
    b = m.INT4Tensor(up(codes), s.to(DEV), up(z) if zeros else None, group)
    off_d, s64 = up(off.astype(np.int32)), s.float().numpy()
    y, tol = Q.grouped(x.double().numpy(), codes, s64, z, group, off, rows)

    def close(got, want, t, what):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= t).all(), f"{what}: worst {np.max(err / np.maximum(t, 1e-300)):.3f} of the bound"

    kw = dict(m_total=M, a_rows=up(rows))
    close(m.int4_grouped_gemv(x.to(DEV), b, off_d, out_dtype=torch.float32, **kw), y, tol + 2.0 ** -24 * np.abs(y) + TINY["f32"], "float32")
    got = m.int4_grouped_gemv(x.to(DEV), b, off_d, **kw)
    assert got.dtype == F[dtype]
    close(got, y, Q.rounded(y, tol, dtype), "16 bit")
    if N % 2 == 0:
        for act in ("silu", "gelu"):
            h, th = Q.gated(y, tol, act)
            close(m.int4_grouped_gemv(x.to(DEV), b, off_d, gated=True, activation=ACT[act], **kw), h, Q.rounded(h, th, dtype), act)
    # rows in place, and behind the last expert: not written
    direct = x.to(DEV)[torch.from_numpy(rows).long().to(DEV)]
    out = torch.full((M + 3, N), 7.0, dtype=F[dtype], device=DEV)
    more = torch.cat([direct, torch.full((3, K), float("nan"), dtype=F[dtype], device=DEV)])
    m.int4_grouped_gemv(more, b, off_d, m_total=M + 3, out=out, max_rows_per_expert_hint=int(max(counts)))
    assert (out[M:] == 7).all()
    close(out[:M], y, Q.rounded(y, tol, dtype), "direct")


@pytest.mark.parametrize("K", [768, 512, 256, 416, 96, 32])
def test_every_hint_gives_the_product(K):
    """The hint picks the kernel, not the result's definition: rows far above and below it."""
    r = np.random.default_rng(3)
    counts = [70, 0, 3, 16, 17]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, N, group = int(off[-1]), 72, 32
    w = m.int4_quantize(up(r.standard_normal((5, N, K)).astype(np.float32)), group, True)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)
    y, tol = Q.grouped(x.double().numpy(), w.codes.cpu().numpy(), w.scales.float().cpu().numpy(), w.zeros.cpu().numpy(), group, off)
    for hint in (0, 1, 16, 17, 64, 10 ** 9):
        got = m.int4_grouped_gemv(x.to(DEV), w, up(off), m_total=M, out_dtype=torch.float32, max_rows_per_expert_hint=hint)
        assert (np.abs(got.double().cpu().numpy() - y) <= tol + 2.0 ** -24 * np.abs(y)).all(), hint


def test_non_finite_rows_and_groups_stay_apart():
    K, N, M = 256, 40, 6
    r = np.random.default_rng(4)
    w = r.standard_normal((1, N, K)).astype(np.float32)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)
    off = up(np.array([0, M], np.int32))
    good = m.int4_grouped_gemv(x.to(DEV), m.int4_quantize(up(w), 64), off, m_total=M)
    x[2, 7], x[4, 200] = float("nan"), float("inf")
    w[0, 5, 70], w[0, 39, 255] = np.inf, np.nan
    got = m.int4_grouped_gemv(x.to(DEV), m.int4_quantize(up(w), 64), off, m_total=M)
    rows, cols = torch.tensor([0, 1, 3, 5]), torch.tensor([c for c in range(N) if c not in (5, 39)])
    assert torch.equal(got.cpu()[rows][:, cols], good.cpu()[rows][:, cols])
    assert torch.isnan(got[:, 5]).all() and torch.isnan(got[:, 39]).all() and torch.isnan(got[2]).all()
    assert not torch.isfinite(got[4]).any()


def test_no_rows():
    b = m.int4_quantize(torch.randn((3, 16, 64), device=DEV), 32)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.randn((5, 64), device=DEV).to(torch.bfloat16)
    assert m.int4_grouped_gemv(x[:0], b, off, m_total=0).shape == (0, 16)
    out = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    m.int4_grouped_gemv(x, b, off, m_total=5, out=out)              # every expert empty
    assert (out == 3).all()


def test_bad_index_arrays_stay_inside():
    """Entries that break their ranges give wrong rows, nothing else (the kernel's own bounds)."""
    b = m.int4_quantize(torch.randn((3, 24, 64), device=DEV), 32)
    x = torch.randn((8, 64), device=DEV).to(torch.bfloat16)
    rows = torch.tensor([0, -5, 8, 2 ** 31 - 1, -2 ** 31, 7, 1, 2], dtype=torch.int32, device=DEV)
    good = torch.where((rows >= 0) & (rows < 8), rows, 0)
    off = torch.tensor([0, 3, 5, 8], dtype=torch.int32, device=DEV)
    a = m.int4_grouped_gemv(x, b, off, m_total=8, a_rows=rows)
    assert torch.equal(a, m.int4_grouped_gemv(x, b, off, m_total=8, a_rows=good))
    for bad in ([0, 5, 3, 8], [-4, 3, 5, 100], [8, 0, 8, 0], [2 ** 31 - 1, -2 ** 31, 0, 5], [0, 8, 0, 8]):
        out = torch.zeros((8, 24), dtype=torch.bfloat16, device=DEV)
        m.int4_grouped_gemv(x, b, torch.tensor(bad, dtype=torch.int32, device=DEV), m_total=8, out=out)
        assert torch.isfinite(out).all()


def test_unaligned_scales():
    """Scales that start 2 bytes behind a border of 16."""
    r = np.random.default_rng(9)
    for group, K in ((32, 1024), (64, 512), (128, 768)):
        w = m.int4_quantize(up(r.standard_normal((2, 50, K)).astype(np.float32)), group, True)
        flat = torch.empty(w.scales.numel() + 1, dtype=w.scales.dtype, device=DEV)
        flat[1:] = w.scales.reshape(-1)
        zf = torch.empty(w.zeros.numel() + 1, dtype=torch.uint8, device=DEV)
        zf[1:] = w.zeros.reshape(-1)
        v = m.INT4Tensor(w.codes, flat[1:].view(w.scales.shape), zf[1:].view(w.zeros.shape), group)
        x = torch.randn((5, K), device=DEV).to(torch.bfloat16)
        off = up(np.array([0, 2, 5], np.int32))
        assert torch.equal(m.int4_grouped_gemv(x, w, off, m_total=5), m.int4_grouped_gemv(x, v, off, m_total=5))
        assert torch.equal(m.int4_dequantize(w), m.int4_dequantize(v))


@pytest.mark.parametrize("N,K", [(1 << 17, 1 << 16)])
def test_weights_above_4_gib(N, K):
    """2^33 codes: offsets past 32 bits; rows of the last columns against a few in float64."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("memory")
    codes = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.rand((1, N, K // 128), device=DEV).to(torch.bfloat16)
    b = m.INT4Tensor(codes, scales, None, 128)
    x = torch.randn((2, K), device=DEV).to(torch.bfloat16)
    y = m.int4_grouped_gemv(x, b, torch.tensor([0, 2], dtype=torch.int32, device=DEV), m_total=2, out_dtype=torch.float32)
    at = [0, N // 2, N - 3, N - 1]
    want, tol = Q.grouped(x.double().cpu().numpy(), codes[:, at].cpu().numpy(), scales[:, at].float().cpu().numpy(), None, 128, [0, 2])
    assert (np.abs(y[:, at].double().cpu().numpy() - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
    v = m.int4_dequantize(b)
    assert torch.equal(v[0, N - 1].double().cpu(), torch.from_numpy(
        Q.round16(Q.dequantize(codes[0, N - 1:].cpu().numpy(), scales[0, N - 1:].float().cpu().numpy(), None, 128)[0].astype(np.float32), "bf16")).double())
    q = m.int4_quantize(v)
    last, sc, _ = Q.quantize(v[0, N - 1:].float().cpu().numpy(), 128, False, "bf16")
    assert np.array_equal(q.codes[0, N - 1:].cpu().numpy(), last)


def test_no_rows_and_rows_of_no_expert():
    w = m.int4_quantize(torch.randn((3, 40, 64), device=DEV), 32, True, torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    for rows in (0, 5):
        x = torch.randn((rows, 64), device=DEV).to(torch.bfloat16)
        assert m.int4_grouped_gemv(x, w, off, m_total=0).shape == (0, 40)
        assert m.int4_grouped_gemv(x, w, off, m_total=0, gated=True).shape == (0, 20)
    # rows that belong to no expert stay as they are
    out = torch.full((5, 40), 3.0, device=DEV)
    m.int4_grouped_gemv(x, w, off, m_total=5, out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("st", ["bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise_whole_range(group, dtype, st, zeros):
    """Groups of any exponent, values of one size or many, quotients on ties; the scale rounds twice, to
    float32 and to its type (7 n 2^-25 by 1/7 is n 2^-25 in float32, halfway between two f16 values)."""
    r = np.random.default_rng(group)
    n = 3000
    e = r.integers(*((-24, 15) if dtype == "f16" else (-140, 126)), (n, 1))
    x = r.standard_normal((n, group)) * np.exp2(e - r.integers(0, 12, (n, group)) * (np.arange(n)[:, None] % 3 == 0))
    h = n // 2
    x[:h] = np.round(x[:h] / np.abs(x[:h]).max(1, keepdims=True) * 14) / 2 * np.exp2(e[:h])
    x[:200, 0] = (15 if zeros else 7) * 2.0 ** -25 * np.arange(200)
    x[:200, 1:] = x[:200, :1] * r.random((200, group - 1))
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x.astype(np.float32)).to(F[dtype])
    got = m.int4_quantize(t.to(DEV), group, zeros, F[st])
    codes, scales, z = Q.quantize(t.float().numpy(), group, zeros, st)
    assert np.array_equal(got.scales.float().cpu().numpy(), scales, equal_nan=True)
    assert np.array_equal(got.codes.cpu().numpy(), codes)
    assert not zeros or np.array_equal(got.zeros.cpu().numpy(), z)
