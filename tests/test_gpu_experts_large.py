"""Operands and results of more than 4 GiB: products, gradients, the gated block
and INT8, at rows and experts on both sides of the limit, against float64."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import experts16 as X
from oracle import int8 as Q
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu
ROWS, WIDE = 262184, 8200          # x 2 bytes: 4.3e9
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _normal(shape, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF, device=DEV).normal_(0, std, generator=g)


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, tol, what):
    err = np.abs(_f64(got) - want)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.3f} of the bound"


def _picked(off):
    """Some rows: the first and last of each expert and around 2^31 and 2^32 bytes of WIDE bf16 values;
    their offsets among the picked."""
    at = {int(b) // (2 * WIDE) + d for b in (2 ** 31, 2 ** 32) for d in (-1, 0, 1)}
    for lo, hi in zip(off[:-1], off[1:]):
        at |= {r for r in (lo, lo + 1, hi - 2, hi - 1)}
    rows = np.array(sorted(r for r in at if 0 <= r < off[-1]))
    return rows, np.searchsorted(rows, off)


@pytest.mark.parametrize("hint", [0, 5000, 200000])
def test_operands(hint):
    """Gathered rows and weights, and the weight gradient."""
    E, N, used = 520, 512, [0, 255, 256, 519]
    print(f"large operands, hint {hint}", flush=True)
    counts = np.zeros(E, int)
    counts[used] = [3, 40, 1, 199]
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    r = np.random.default_rng(7)
    rows = r.integers(ROWS - 5000, ROWS, M)
    rows[::3] = r.integers(0, ROWS, len(rows[::3]))
    rows[-1] = ROWS - 1
    a, b, dy = _normal((ROWS, WIDE), 1), _normal((E, N, WIDE), 2, 0.02), _normal((M, N), 3)
    off_d, rows_d = up(off.astype(np.int32)), up(rows.astype(np.int32))
    y = m.moe_grouped_gemm(a, b, off_d, m_total=M, a_rows=rows_d, max_rows_per_expert_hint=hint)
    da, db = m.moe_grouped_gemm_backward(dy, a, b, off_d, a_rows=rows_d, max_rows_per_expert_hint=hint)
    a64, b64 = _f64(a[torch.from_numpy(rows).to(DEV)]), _f64(b[used])
    small = np.concatenate([[0], np.cumsum(counts[used])])
    _close(y, *X.product(a64, b64, small), "y")
    (rda, tda), (rdb, tdb) = X.product_grad(_f64(dy), a64, b64, small)
    _close(da, rda, tda, "da")
    _close(db[used], rdb, tdb, "db")
    for e in range(E):
        if e not in used:
            assert not db[e].any(), e


def test_results_and_row_gradients():
    """y and dy of 4.3e9 bytes, then da."""
    print("large results", flush=True)
    off, K = np.array([0, 100000, 100000, ROWS - 14]), 64
    off_d, (rows, small) = up(off.astype(np.int32)), _picked(off)
    at = torch.from_numpy(rows).to(DEV)
    a, b = _normal((ROWS, K), 4), _normal((3, WIDE, K), 5, 0.1)
    y = torch.full((ROWS, WIDE), 7.0, dtype=BF, device=DEV)
    m.moe_grouped_gemm(a, b, off_d, m_total=ROWS, out=y)
    _close(y[at], *X.product(_f64(a[at]), _f64(b), small), "y")
    assert (y[ROWS - 14:] == 7).all()
    y.normal_(0, 1, generator=torch.Generator(device=DEV).manual_seed(6))
    da, db = m.moe_grouped_gemm_backward(y, a, b, off_d)
    _close(da[at], *X.product_grad(_f64(y[at]), _f64(a[at]), _f64(b), small)[0], "da")
    cols = [0, 1, 4099, WIDE - 1]
    _close(db[:, cols], *X.product_grad(_f64(y[:, cols]), _f64(a), _f64(b[:, cols]), off)[1], "db")
    # the wide side as the gradient of the rows
    b = b.transpose(1, 2).contiguous()
    dy = a
    y.fill_(7.0)
    m.moe_grouped_gemm_backward(dy, torch.empty((ROWS, WIDE), dtype=BF, device=DEV), b, off_d, need_db=False, da=y)
    b64 = _f64(b)
    want, tol = X.product_grad(_f64(dy[at]), np.zeros((len(rows), WIDE)), b64, small)[0]
    _close(y[at], want, tol, "wide da")
    assert (y[ROWS - 14:] == 7).all()


def test_gated_block():
    """Saved pre-activations of 8.6e9 bytes, and a workspace of as many."""
    print("large gated block", flush=True)
    H, I, off = 64, 4104, np.array([0, 100001, ROWS - 14])
    off_d, (rows, small) = up(off.astype(np.int32)), _picked(off)
    at = torch.from_numpy(rows).to(DEV)
    x, w, dh = _normal((ROWS, H), 8), _normal((2, 2 * I, H), 9, 0.1), _normal((ROWS, I), 10)
    h, gu = m.moe_gated_ffn(x, w, off_d, m_total=ROWS, save_gu=True)
    dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off_d)
    (rh, th), (rgu, tgu) = X.gated(_f64(x[at]), _f64(w), small)
    _close(h[at], rh, th, "h")
    _close(gu[at], rgu, tgu, "gu")
    _close(dx[at], *X.gated_grad(_f64(dh[at]), _f64(x[at]), _f64(w), small)[0], "dx")
    cols = np.array([0, 2047, I - 1])
    both = np.concatenate([cols, I + cols])
    _close(dw[:, both], *X.gated_grad(_f64(dh[:, cols]), _f64(x), _f64(w[:, both]), off)[1], "dw")


def test_int8():
    """Codes of rows and weights, and float32 results."""
    print("large int8", flush=True)
    R, E, N, K, used = 524320, 520, 1024, 8208, [0, 255, 256, 519]
    counts = np.zeros(E, int)
    counts[used] = [3, 40, 1, 60]
    off = np.concatenate([[0], np.cumsum(counts)])
    M, r = int(off[-1]), np.random.default_rng(11)
    rows = r.integers(R - 5000, R, M)
    rows[::3], rows[-1] = r.integers(0, R, len(rows[::3])), R - 1
    g = torch.Generator(device=DEV).manual_seed(12)
    a = torch.empty((R, K), dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    b = torch.empty((E, N, K), dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    sa, sb = up((r.random(R) + 0.5).astype(np.float32)), up((r.random((E, N)) + 0.5).astype(np.float32))
    small = np.concatenate([[0], np.cumsum(counts[used])])
    at = torch.from_numpy(rows).to(DEV)
    want, tol = Q.grouped_gemm(a[at].cpu().numpy(), sa[at].cpu().numpy(), b[used].cpu().numpy(), sb[used].cpu().numpy(), small)
    for hint in (0, 5000, 200000):
        y = m.int8_grouped_gemm(m.INT8Tensor(a, sa), m.INT8Tensor(b, sb), up(off.astype(np.int32)), m_total=M,
                                a_rows=up(rows.astype(np.int32)), epilogue=m.EPI_F32, max_rows_per_expert_hint=hint)
        _close(y, want, tol, f"y, hint {hint}")
    del a, b
    off = np.array([0, 100001, ROWS - 14])
    rows, small = _picked(off)
    at = torch.from_numpy(rows).to(DEV)
    a = torch.empty((ROWS, 64), dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    b = torch.empty((2, 4112, 64), dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    sb = up((r.random((2, 4112)) + 0.5).astype(np.float32))
    sa = sa[:ROWS].contiguous()
    y = m.int8_grouped_gemm(m.INT8Tensor(a, sa), m.INT8Tensor(b, sb), up(off.astype(np.int32)), m_total=ROWS, epilogue=m.EPI_F32)
    _close(y[at], *Q.grouped_gemm(a[at].cpu().numpy(), sa[at].cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy(), small), "wide y")


def test_int8_quantizer():
    print("large quantiser", flush=True)
    R, C = 524320, 8208
    x = _normal((R, C), 13)
    q = m.int8_quantize(x)
    at = [0, 1, 2 ** 31 // C, 2 ** 31 // (2 * C), 2 ** 32 // C, 2 ** 32 // C + 1, R - 1]
    codes, scales = Q.quantize(x[at].float().cpu().numpy())
    assert np.array_equal(q.codes[at].cpu().numpy(), codes) and np.array_equal(q.scales[at].cpu().numpy(), scales)
