"""Renormalised weights of chosen experts whose logits lie far below those of experts
that were looked at and not chosen: the choice is by keys with a bias, where such
logits tie, and the weights are the chosen scores' shares whatever the others hold."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import router as R
from tests.gpu_common import DEV, up
from tests.test_gpu_router import F, KIND, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 2100])
@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 2, 1)], ids=str)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_chosen_far_below_others_that_tie(kind, groups, k, T, dtype):
    """Experts 1 to 3 of logits -1000, -1002, -1004 and 4 to 7 of -100 share the key 1 (their scores are below
    float64's step there): the lower ids are chosen."""
    E = 64
    r = np.random.default_rng(k)
    l = np.tile(r.standard_normal(E).astype(np.float32), (T, 1))
    l[:, 1:4] = [-1000, -1002, -1004]
    l[:, 4:8] = -100
    bias = np.full(E, -1, np.float32)
    bias[1:8] = 1
    t = torch.from_numpy(l).to(F[dtype])
    ids, w, _, _ = R.route(t.double().numpy(), k, kind, bias, *groups, True, 2.5)
    assert (ids == np.arange(1, k + 1)).all() and abs(w.sum() - 2.5 * T) < 1e-9 * T
    got = m.moe_route_scored(t.to(DEV), k, score=KIND[kind], bias=up(bias), n_group=groups[0], topk_group=groups[1],
                             group_top=groups[2], scale=2.5)
    assert np.array_equal(got.topk_ids.cpu().numpy(), ids)
    gw = got.topk_w.double().cpu().numpy()
    # float64 until one rounding to float32 (and 2^-40 for the float64 steps)
    assert (np.abs(gw - w) <= w * U * (1 + 2.0 ** -15)).all(), (gw[0], w[0])
