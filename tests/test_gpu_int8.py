"""INT8 quantiser and grouped product against oracle/int8.py: codes and scales
bit for bit, products within three float32 roundings of exact integer sums."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import int8 as Q
from oracle.experts16 import U
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 24), (5, 256), (37, 6144), (2, 520), (130, 1000), (2, 8200), (1, 40008)])
def test_quantize_bits(rows, cols, dtype):
    print(f"int8 quantize {rows}x{cols} {dtype}", flush=True)
    r = np.random.default_rng([rows, cols])
    x = (r.standard_normal((rows, cols)) * 10.0 ** r.integers(-6, 6, (rows, 1))).astype(np.float32)
    if rows > 1:
        x[1] = 0                                    # scale 1, codes 0
    if rows > 2:
        x[2, :] = np.where(np.arange(cols) % 2, 1e-45, 0)   # absmax / 127 rounds to 0: scale 1
    if rows > 3:
        k = np.arange(cols) % 255 - 127             # every code and every tie between two
        x[3] = k + 0.5 * (np.arange(cols) % 2) * (np.abs(k) < 127)
        x[3, 0] = 127
    t = torch.from_numpy(x)
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    q = m.int8_quantize(t.to(DEV))
    codes, scales = Q.quantize(t.float().numpy())
    assert np.array_equal(q.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_quantize_dense_quotients():
    """Every rounding decision near a tie: quotients k + 1/2 moved by a few
    float32 steps, for many scales (the division has to be the correctly
    rounded one)."""
    r = np.random.default_rng(6)
    rows, cols = 512, 1024
    top = (2.0 ** r.uniform(-20, 20, rows)).astype(np.float32)
    s = (top * np.float32(1 / 127)).astype(np.float32)
    k = r.integers(-126, 126, (rows, cols)) + 0.5
    x = (k * s[:, None].astype(np.float64)).astype(np.float32)
    x = (x.view(np.int32) + r.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    x[:, 0] = top
    q = m.int8_quantize(up(x))
    codes, scales = Q.quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


GROUPS = [([1], 64, 32), ([0, 1, 0, 2], 48, 144), ([8] * 5, 256, 128), ([17, 0, 63, 65], 272, 80), ([129, 5], 16, 16),
          ([257, 31, 1, 0, 16], 512, 256), ([520], 336, 272), ([3, 700, 0, 64], 192, 1040),
          # few rows an expert, short reductions, many tiles: the 64-row tiles
          ([5] * 30 + [0, 70, 0, 129, 64] + [9] * 6, 2080, 144), ([5] * 30 + [0, 70, 0, 129, 64] + [9] * 6, 1040, 16)]


@pytest.mark.parametrize("counts,N,K", GROUPS, ids=[f"{'-'.join(map(str, c)) if len(c) < 9 else f'{len(c)}experts'}x{n}x{k}" for c, n, k in GROUPS])
def test_grouped_product(counts, N, K):
    print(f"int8 product {counts} N={N} K={K}", flush=True)
    r = np.random.default_rng([N, K])
    off = np.concatenate([[0], np.cumsum(counts)])
    M, E, T = int(off[-1]), len(counts), 64
    a, b = r.integers(-127, 128, (T, K)).astype(np.int8), r.integers(-127, 128, (E, N, K)).astype(np.int8)
    sa = (r.random(T) * 0.1 + 1e-3).astype(np.float32)
    sb = (r.random((E, N)) * 1e-3 + 1e-5).astype(np.float32)
    rows = r.integers(0, T, M).astype(np.int32)
    A, B = m.INT8Tensor(up(a), up(sa)), m.INT8Tensor(up(b), up(sb))
    kw = dict(m_total=M, a_rows=up(rows))
    off_d = up(off.astype(np.int32))
    y, tol = Q.grouped_gemm(a, sa, b, sb, off, rows)

    def close(got, want, t, what):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= t).all(), f"{what}: worst {np.max(err / np.maximum(t, 1e-300)):.3f} of the bound"

    for hint in (0, 5000, 200000):
        close(m.int8_grouped_gemm(A, B, off_d, epilogue=m.EPI_F32, max_rows_per_expert_hint=hint, **kw), y, tol, "f32")
        close(m.int8_grouped_gemm(A, B, off_d, max_rows_per_expert_hint=hint, **kw), y, Q.rounded(y, tol, "bf16"), "bf16")
        h, th = Q.swiglu(y, tol)
        close(m.int8_grouped_gemm(A, B, off_d, epilogue=m.EPI_SWIGLU_BF16, max_rows_per_expert_hint=hint, **kw), h,
              Q.rounded(h, th, "bf16"), "swiglu")
    # direct rows
    d = m.INT8Tensor(up(a[rows]), up(sa[rows]))
    assert torch.equal(m.int8_grouped_gemm(d, B, off_d, m_total=M), m.int8_grouped_gemm(A, B, off_d, **kw))


def test_extreme_codes_and_longest_sum():
    """K = 131056 of codes -128 and 127: the exact sum reaches 2^31 - 2^18."""
    K, N = 131056, 16
    a = np.full((2, K), -128, np.int8)
    a[1] = 127
    b = np.full((1, N, K), -128, np.int8)
    b[0, 1::2] = 127
    one, ones = np.ones(2, np.float32), np.ones((1, N), np.float32)
    off = np.array([0, 2])
    y, tol = Q.grouped_gemm(a, one, b, ones, off)
    got = m.int8_grouped_gemm(m.INT8Tensor(up(a), up(one)), m.INT8Tensor(up(b), up(ones)), up(off.astype(np.int32)),
                              m_total=2, epilogue=m.EPI_F32).double().cpu().numpy()
    assert (np.abs(got - y) <= U * np.abs(y)).all() and y.max() == 128 * 128 * K


def test_rows_behind_the_last_expert_keep_their_bytes():
    r = np.random.default_rng(3)
    a, b = r.integers(-127, 128, (40, 64)).astype(np.int8), r.integers(-127, 128, (2, 32, 64)).astype(np.int8)
    sa = np.full(40, np.nan, np.float32)          # scales behind the last expert are not used
    sa[:33] = 0.5
    A, B = m.INT8Tensor(up(a), up(sa)), m.INT8Tensor(up(b), up(np.ones((2, 32), np.float32)))
    for hint in (4, 5000, 200000):
        out = torch.full((40, 32), 7.0, dtype=torch.bfloat16, device=DEV)
        m.int8_grouped_gemm(A, B, up(np.array([0, 12, 33], np.int32)), m_total=40, out=out, max_rows_per_expert_hint=hint)
        assert (out[33:] == 7).all() and torch.isfinite(out.float()).all()


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        m.int8_quantize(x.half())
    with pytest.raises(ValueError):
        m.int8_quantize(x.t())
    with pytest.raises(m.NVFP4MoEError):
        m.int8_quantize(x[:, :12].contiguous())
    q = m.int8_quantize(x)
    w = m.int8_quantize(torch.ones((2, 32, 64), device=DEV))
    assert w.scales.shape == (2, 32)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for kw, err in ((dict(epilogue=m.EPI_COMBINE_F32), ValueError), (dict(m_total=5), ValueError),
                    (dict(out=torch.empty((4, 16), dtype=torch.bfloat16, device=DEV)), ValueError),
                    (dict(out=torch.empty((4, 32), device=DEV)), TypeError)):
        with pytest.raises(err):
            m.int8_grouped_gemm(q, w, off, **{"m_total": 4, **kw})
    with pytest.raises(TypeError):
        m.int8_grouped_gemm(m.INT8Tensor(q.codes.to(torch.uint8), q.scales), w, off, m_total=4)
    with pytest.raises(ValueError):
        m.int8_grouped_gemm(m.INT8Tensor(q.codes, q.scales[:3].contiguous()), w, off, m_total=4)
