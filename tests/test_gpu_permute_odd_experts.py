"""The permutation with numbers of experts that are no multiple of 4, around the sizes
where a thread's part of the histograms ends inside or behind a batch of them: rows
exactly as oracle/moe.py has them."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import moe as OM
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunks", [1, 2, 7, 8, 9, 16, 17, 33, 65])
@pytest.mark.parametrize("E", [5, 62, 129, 257, 511, 513, 1023, 1025, 2049, 4095])
def test_chunks_around_a_batch(E, chunks):
    n = 1024 * chunks - chunks % 3
    r = np.random.default_rng([E, chunks])
    ids = r.integers(0, E, n)
    ids[: n // 4] = E - 1                       # a hot expert
    l = torch.zeros((n, E), dtype=torch.bfloat16, device=DEV)
    l[torch.arange(n, device=DEV), up(ids)] = 2.0
    counts, offsets, src, row_of, _ = OM.permute(ids[:, None], np.ones((n, 1), np.float32), E)
    got = m.moe_route_scored(l, 1)
    assert np.array_equal(got.topk_ids.cpu().numpy()[:, 0], ids)
    for a, b in ((got.counts, counts), (got.offsets, offsets), (got.perm_src_token, src), (got.perm_of_assignment, row_of)):
        assert np.array_equal(a.cpu().numpy(), b)
