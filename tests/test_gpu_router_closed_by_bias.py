"""A bias of -inf or NaN closes an expert to the choice and to nothing else: its score,
its share of a softmax's sum and its logit's gradient remain.  Values written out by hand."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from tests.gpu_common import up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T", [1, 40, 4100])
@pytest.mark.parametrize("closed", [-np.inf, np.nan])
def test_softmax(closed, T):
    l = up(np.tile(np.array([0, 0, 0, 0], np.float32), (T, 1)))
    bias = up(np.array([0, closed, 0.5, 0], np.float32))
    r, s = m.moe_route_scored(l, 2, bias=bias, renormalize=False, scale=2.0, save_scores=True)
    assert (r.topk_ids.cpu() == torch.tensor([2, 0], dtype=torch.int32)).all()
    # quarters and halves of exactly equal exponentials: exact
    assert (s == 0.25).all() and (r.topk_w == 0.5).all()
    r = m.moe_route_scored(l, 2, bias=bias, scale=2.0)
    assert (r.topk_w == 1.0).all()
    # all three open ones and the closed one behind them, with weight 0
    r = m.moe_route_scored(l, 4, bias=bias, renormalize=False)
    assert (r.topk_ids.cpu() == torch.tensor([2, 0, 3, 1], dtype=torch.int32)).all()
    assert (r.topk_w.cpu() == torch.tensor([0.25, 0.25, 0.25, 0])).all()
    # dL/ds = (0, 1, 0, 0): s (q - sum s q)
    dw = up(np.tile(np.array([0, 0], np.float32), (T, 1)))
    ids = up(np.tile(np.array([2, 0], np.int32), (T, 1)))
    q = up(np.array([0, 1, 0, 0], np.float32))
    d = m.moe_route_scored_backward(dw, l, ids, bias=bias, renormalize=False, d_scores=q).double().cpu().numpy()
    # each term from a score of a few half steps and four sums
    assert (np.abs(d - np.array([-1, 3, -1, -1]) / 16) <= 16 * U).all()
    dw[:, 0] = 1.0
    d = m.moe_route_scored_backward(dw, l, ids, bias=bias, renormalize=False).double().cpu().numpy()
    assert (np.abs(d - np.array([-1, -1, 3, -1]) / 16) <= 16 * U).all()


@pytest.mark.parametrize("T", [1, 40, 4100])
@pytest.mark.parametrize("closed", [-np.inf, np.nan])
def test_sigmoid(closed, T):
    l = up(np.tile(np.array([0, 0, 0, 0], np.float32), (T, 1)))
    bias = up(np.array([0, closed, 0.5, 0], np.float32))
    r, s = m.moe_route_scored(l, 4, score=m.SCORE_SIGMOID, bias=bias, renormalize=False, save_scores=True)
    assert (r.topk_ids.cpu() == torch.tensor([2, 0, 3, 1], dtype=torch.int32)).all()
    assert (s == 0.5).all() and (r.topk_w.cpu() == torch.tensor([0.5, 0.5, 0.5, 0])).all()
    # the closed expert's weight has no gradient, its score has: (1 - s) s q
    dw = up(np.tile(np.array([0, 0, 0, 1], np.float32), (T, 1)))
    q = up(np.array([0, 1, 0, 0], np.float32))
    d = m.moe_route_scored_backward(dw, l, r.topk_ids, score=m.SCORE_SIGMOID, bias=bias, renormalize=False, d_scores=q)
    assert (np.abs(d.double().cpu().numpy() - np.array([0, 0.25, 0, 0])) <= 8 * U).all()
