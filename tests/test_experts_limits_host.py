"""Host-side checks (no GPU needed) at the size limits that the header states
for the 16-bit experts' gradients: beyond them a call is refused before
anything is enqueued, and its workspace query returns 0."""
import ctypes

import pytest

import block_scaled_fp4_permute_amd as m

try:
    import torch
    _HAVE_GPU = torch.cuda.is_available()
except Exception:  # pragma: no cover
    _HAVE_GPU = False
pytestmark = pytest.mark.skipif(_HAVE_GPU, reason="fake device addresses: host-only checks, run without a GPU")

F = 1 << 20            # aligned, never dereferenced


@pytest.mark.parametrize("E,I,m_total", [(1, 8, 2 ** 30 - 1), (1, 64, 2 ** 30 - 512), (4096, 8, 2 ** 30 - 2 ** 18),
                                         (1, 72, 2 ** 29), (4, 2 ** 20, 2 ** 16)])
def test_activation_gradient_of_too_many_blocks(E, I, m_total):
    """2^24 workgroups of 64 rows and 64 columns, which no grid holds."""
    args = m.GatedGradArgs(x=F, dtype=m.BF16, a_rows=None, x_rows=m_total, w=F, offsets=F, E=E, H=8, I=I, m_total=m_total,
                           activation=0, max_rows_per_expert_hint=0, gu=F, dh=F, dx=F, dw=F)
    assert m.lib().moe_gated_ffn_backward(ctypes.byref(args), F, 2 ** 63, None) == m.ERR_UNSUPPORTED
    assert m.lib().moe_gated_ffn_backward_workspace_size(E, 8, I, m_total) == 0


@pytest.mark.parametrize("E,I,m_total", [(1, 8, 2 ** 30 - 576), (4096, 64, 2 ** 30 - 2 ** 18 - 512), (1, 128, 2 ** 29 - 576)])
def test_the_largest_sizes_have_a_workspace(E, I, m_total):
    assert m.lib().moe_gated_ffn_backward_workspace_size(E, 8, I, m_total) > 0


def _gated_grad(E, H, I, M):
    args = m.GatedGradArgs(x=F, dtype=m.BF16, a_rows=None, x_rows=M, w=F, offsets=F, E=E, H=H, I=I, m_total=M, activation=0,
                           max_rows_per_expert_hint=0, gu=F, dh=F, dx=F, dw=F)
    return m.lib().moe_gated_ffn_backward(ctypes.byref(args), None, 0, None)


def _product_grad(E, N, K, M):
    args = m.ProductGradArgs(a=F, dtype=m.BF16, a_rows=None, a_rows_total=M, b=F, offsets=F, E=E, N=N, K=K, m_total=M,
                             max_rows_per_expert_hint=0, dy=F, da=F, db=F)
    return m.lib().moe_grouped_gemm_backward(ctypes.byref(args), None, 0, None)


@pytest.mark.parametrize("E,N,K,M", [
    (4096, 2 ** 20, 2 ** 20, 16),           # 2^31 tiles of a weight gradient
    (1, 2 ** 26, 2 ** 26, 2 ** 20), (1, 2 ** 20, 64, 2 ** 29), (4, 64, 2 ** 26 + 8, 16), (4, 2 ** 26 + 8, 64, 16),
    (4, 64, 60, 16), (4097, 64, 64, 16), (4, 64, 64, 2 ** 30)])
def test_queries_return_0_for_sizes_that_the_calls_refuse(E, N, K, M):
    """Without a workspace: a call on sizes that have one would ask for it."""
    if N % 16 == 0:
        assert _gated_grad(E, K, N // 2, M) in (m.ERR_INVALID, m.ERR_UNSUPPORTED)
        assert m.lib().moe_gated_ffn_backward_workspace_size(E, K, N // 2, M) == 0
    assert _product_grad(E, N, K, M) in (m.ERR_INVALID, m.ERR_UNSUPPORTED)
    assert m.lib().moe_grouped_gemm_backward_workspace_size(E, N, K, M) == 0
