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
