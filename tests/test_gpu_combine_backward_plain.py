"""Gradients of the combine without weights (a plain sum of each token's rows): every row's
is its token's, and those of weights that all are 1."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (7, 3, 520), (300, 8, 2056)])
def test_plain_sum(T, k, H, dtype):
    g = torch.Generator(device=DEV).manual_seed(T)
    dout, y = (torch.randn(s, generator=g, device=DEV).to(dtype) for s in ((T, H), (T * k, H)))
    rows = np.random.default_rng(T).permutation(T * k).astype(np.int32)
    perm = up(rows)
    dy, dw = m.moe_unpermute_combine_backward(dout, y, perm, None, k=k)
    assert torch.equal(dy[perm.long()].view(T, k, H), dout[:, None].expand(T, k, H))
    for got, want in zip((dy, dw), m.moe_unpermute_combine_backward(dout, y, perm, torch.ones((T, k), device=DEV))):
        assert torch.equal(got, want)
    dy, dw2 = m.moe_unpermute_combine_backward(dout, y[perm.long()].contiguous(), None, None, k=k)
    assert torch.equal(dy.view(T, k, H), dout[:, None].expand(T, k, H)) and torch.equal(dw2, dw)
    # and the forward call's: out = sum of the rows
    out = m.moe_unpermute_combine(y, perm, None, T, k, out_dtype=torch.float32)
    want = y[perm.long()].view(T, k, H).double().sum(1)
    assert ((out.double() - want).abs() <= k * 2.0 ** -24 * y.abs().max().double() * k).all()
