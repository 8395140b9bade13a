"""int8_quantize on rows that hold a NaN or an infinity: scale NaN and codes 0,
so that everything computed from such a row is NaN, and no other row changes."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import int8 as Q
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
# a row length for each form of the kernel
@pytest.mark.parametrize("cols", [8, 504, 1000, 2048, 4096, 6144, 8192, 16384, 20000])
def test_rows_with_nan_or_infinity(cols, dtype):
    print(f"int8 quantize, not finite: {cols} {dtype}", flush=True)
    r = np.random.default_rng(cols)
    x = r.standard_normal((11, cols)).astype(np.float32)
    x[9] = 0
    t = torch.from_numpy(x)
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    clean = t.clone()
    bad = {1: np.nan, 3: np.inf, 4: -np.inf, 7: np.nan, 10: -np.nan}
    for row, v in bad.items():
        t[row, int(r.integers(0, cols))] = float(v)
    t[7, cols - 1] = float("inf")
    q = m.int8_quantize(t.to(DEV))
    codes, scales = Q.quantize(clean.float().numpy())
    rows = sorted(bad)
    codes[rows], scales[rows] = 0, np.nan
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales, equal_nan=True)


def test_a_product_shows_them():
    """Its rows alone are NaN, in each epilogue."""
    x = torch.ones((6, 64), dtype=torch.bfloat16, device=DEV)
    x[2, 5], x[4, 63] = float("nan"), float("inf")
    a, b = m.int8_quantize(x), m.int8_quantize(torch.ones((2, 32, 64), device=DEV))
    off = up(np.array([0, 3, 6], np.int32))
    for epi in (m.EPI_F32, m.EPI_BF16, m.EPI_SWIGLU_BF16):
        for hint in (0, 5000, 200000):
            y = m.int8_grouped_gemm(a, b, off, m_total=6, epilogue=epi, max_rows_per_expert_hint=hint)
            assert torch.isnan(y).all(1).tolist() == [False, False, True, False, True, False]
            assert torch.isfinite(y[[0, 1, 3, 5]]).all()


def test_largest_finite_values_stay():
    top = np.finfo(np.float32).max
    x = np.array([[top, -top, top / 2, 0, 1, -1, top / 254, 3]], np.float32)
    q = m.int8_quantize(up(x))
    codes, scales = Q.quantize(x)
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
