"""The router's choice where float32 keys run out, by thousands of tokens, and the
permutation around the sizes where it changes kernels: ids and rows exactly as
oracle/router.py and oracle/moe.py have them."""
import itertools

import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import moe as OM
from oracle import router as R
from tests.gpu_common import DEV, up
from tests.test_gpu_router import F, KIND, _call, _check, _edge_rows, _logits, _want

pytestmark = pytest.mark.gpu


def _clusters(T, E, k, seed):
    """Rows with `size` experts a few float32 steps apart, the k-th among them or just behind or before them."""
    r = np.random.default_rng(seed)
    l = r.standard_normal((T, E)).astype(np.float32)
    for t in range(T):
        size = int(r.integers(2, min(E, 48) + 1))
        above = int(r.integers(max(0, k - size - 1), k + 2))           # experts clearly above the cluster
        at = r.permutation(E)
        center = np.float32([2.5, -2.5, 0.125][t % 3])
        l[t, at[above:above + size]] = (center.view(np.uint32) + r.integers(0, [2, 5, 40][t // 3 % 3], min(size, E - above)).astype(np.uint32)).view(np.float32)
        l[t, at[:above]] = 4.0 + r.random(min(above, E)).astype(np.float32)
        rest = at[above + size:]
        l[t, rest] = -4.0 + r.random(len(rest)).astype(np.float32)
    return l


def _other_groups(row, ids, k, kind, bias, groups):
    """Whether ids follow from groups whose values float64 cannot tell from the oracle's: e^a + e^b
    and e^c + e^d with a + b = c + d differ by ((a - b)^2 - (c - d)^2) / 4 relative, which for logits
    a few steps of 2^-26 apart is below 2^-53, under the rounding of either sum.  A value is
    the sum of two scores of up to 6 half steps (exponential, quotient, bias): within 16 of them."""
    n, keep, top = groups
    key = R.scores(row[None], kind)[0][0] + (0 if bias is None else bias.astype(np.float64))
    order = row if bias is None else key
    value = np.sort(key.reshape(n, -1), 1)[:, -top:].sum(1)
    last = np.sort(value)[-keep]
    far = 16 * 2.0 ** -53 * np.abs(key).max()
    sure, maybe = np.flatnonzero(value > last + far), np.flatnonzero(np.abs(value - last) <= far)
    for more in itertools.combinations(maybe, keep - len(sure)):
        stays = np.isin(np.arange(len(row)) // (len(row) // n), np.concatenate([sure, more]))
        if sorted(np.flatnonzero(stays), key=lambda e: (-order[e], e))[:k] == ids.tolist():
            return True
    return False


def _same(got, l, k, kind, bias, groups, E):
    ids, w, _, o = R.route(l, k, kind, bias, *groups, True, 1.0)
    g = got.topk_ids.cpu().numpy()
    odd = np.flatnonzero((g != ids).any(1))
    for t in odd:
        assert groups[0] > 1 and _other_groups(l[t], g[t], k, kind, bias, groups), (t, g[t], ids[t])
    gw = got.topk_w.cpu().numpy()
    same = np.setdiff1d(np.arange(len(l)), odd)
    assert len(odd) <= 0.02 * len(l)
    assert (np.abs(gw - w) <= np.abs(w) * 2.0 ** -24 * (1 + 2.0 ** -15))[same].all()


@pytest.mark.parametrize("bias", ["none", "zero", "steps"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2), (16, 3, 1)], ids=str)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(500, 256, 8), (2100, 256, 8), (2100, 64, 4), (2100, 192, 9), (300, 1024, 32)])
def test_clusters_of_neighbouring_keys(T, E, k, kind, groups, bias):
    print("clusters", T, E, k, kind, groups, bias, flush=True)
    l = _clusters(T, E, k, T + E)
    b = None
    if bias != "none":
        b = np.zeros(E, np.float32)
        if bias == "steps":
            b[::3], b[1::5] = 2.0 ** -24, -(2.0 ** -23)
    got = m.moe_route_scored(up(l), k, score=KIND[kind], bias=None if b is None else up(b), n_group=groups[0],
                             topk_group=groups[1], group_top=groups[2])
    _same(got, l.astype(np.float64), k, kind, b, groups, E)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T", [64, 4096])
def test_few_values_many_ties(T, bias, groups, dtype):
    r = np.random.default_rng(T)
    l = torch.from_numpy((r.integers(-3, 4, (T, 256)) / 4).astype(np.float32)).to(F[dtype])
    l[::7] = 0                                  # padding: every expert alike
    b = (r.integers(0, 2, 256) / 8).astype(np.float32) if bias else None
    got = m.moe_route_scored(l.to(DEV), 8, score=m.SCORE_SIGMOID, bias=None if b is None else up(b), n_group=groups[0],
                             topk_group=groups[1], group_top=groups[2])
    _same(got, l.double().numpy(), 8, "sigmoid", b, groups, 256)


@pytest.mark.parametrize("n", [1023, 1024, 1025, 262143, 262144, 262145])
@pytest.mark.parametrize("E", [3, 61, 256, 4096])
def test_permutation_around_its_sizes(E, n):
    """One expert a token: chunks of 1024 assignments, one kernel more beyond 256 of them."""
    r = np.random.default_rng([E, n])
    l = torch.zeros((n, E), device=DEV)
    ids = r.integers(0, E, n)
    ids[: n // 3] = E - 1                       # a hot expert
    l[torch.arange(n, device=DEV), up(ids)] = 2.0
    counts, offsets, src, row_of, _ = OM.permute(ids[:, None], np.ones((n, 1), np.float32), E)
    for got in (m.moe_route_permute(l, 1), m.moe_route_scored(l, 1)):
        assert np.array_equal(got.topk_ids.cpu().numpy()[:, 0], ids)
        for a, b in ((got.counts, counts), (got.offsets, offsets), (got.perm_src_token, src), (got.perm_of_assignment, row_of)):
            assert np.array_equal(a.cpu().numpy(), b)
        assert (got.perm_weight == 1).all()
        del got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T", [5, 64, 2100])
def test_zeros_of_either_sign_are_one_value(T, bias, groups, dtype):
    r = np.random.default_rng(T)
    l = torch.from_numpy(np.where(r.random((T, 64)) < 0.5, np.float32(-0.0), np.float32(0.0))).to(F[dtype])
    l[::3, ::9] = 1.0
    b = np.where(r.random(64) < 0.5, np.float32(-0.0), np.float32(0.0)).astype(np.float32) if bias else None
    got = m.moe_route_scored(l.to(DEV), 6, score=m.SCORE_SIGMOID, bias=None if b is None else up(b), n_group=groups[0],
                             topk_group=groups[1], group_top=groups[2])
    _same(got, l.double().numpy(), 6, "sigmoid", b, groups, 64)


@pytest.mark.parametrize("c", [
    (4095, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),        # the last on 64 lanes a token with scores
    (4096, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),
    (4099, 256, 16, "softmax", False, (1, 1, 1), False, "bf16"),
    (4101, 61, 5, "softmax", True, (1, 1, 1), True, "f16"),
    (4097, 96, 6, "sigmoid", True, (12, 4, 2), False, "f32"),
    (4098, 250, 8, "softmax", True, (5, 3, 1), False, "f32"),
], ids=str)
def test_scores_of_many_tokens(c):
    _, t, l, bias = _logits(c)
    got, scores = _call(t, c, bias, save_scores=True)
    _check(got, scores, _want(l, c, bias), c[2], c[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 2)], ids=str)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_edge_rows_of_many_tokens(bias, kind, groups, dtype):
    t = torch.from_numpy(_edge_rows(72, dtype != "f32")).to(F[dtype])
    b = None
    if bias:
        b = (np.random.default_rng(3).standard_normal(72) * 0.01).astype(np.float32)
        b[3], b[5], b[9] = -np.inf, np.nan, np.inf
    for renormalize in (True, False):
        c = (len(t), 72, 6, kind, bias, groups, renormalize, dtype)
        ids, w, s, _ = _want(t.double().numpy(), c, b)
        got, scores = _call(t.repeat(200, 1), c, b, save_scores=True)
        _check(got, scores, (np.tile(ids, (200, 1)), np.tile(w, (200, 1)), np.tile(s, (200, 1)), None), 6, 72)


@pytest.mark.parametrize("T", [5, 300, 2100, 4100])
@pytest.mark.parametrize("weights", [True, False], ids=["perm_weight", "none"])
def test_given_outputs(T, weights):
    """Results, scores and a workspace of the caller's, four bytes off any alignment and between guards;
    the workspace holds another call's rest."""
    E, k = 64, 4
    c = (T, E, k, "sigmoid", True, (8, 4, 2), True, "f32")
    _, t, l, bias = _logits(c)
    guard = []

    def block(*shape, dtype=torch.int32):
        n = int(np.prod(shape))
        whole = torch.full((n + 12,), 77, dtype=dtype, device=DEV)
        guard.append((whole, n))
        return whole[5:5 + n].view(shape)

    out = m.Routing(block(T, k), block(T, k, dtype=torch.float32), block(E), block(E + 1), block(T * k), block(T * k),
                    block(T * k, dtype=torch.float32) if weights else None)
    scores = block(T, E, dtype=torch.float32)
    ws = torch.full((m.lib().moe_route_permute_workspace_size(T, E, k),), 255, dtype=torch.uint8, device=DEV)
    x = block(T, E, dtype=torch.float32)
    x.copy_(t)
    got, s = m.moe_route_scored(x, k, score=m.SCORE_SIGMOID, bias=up(bias), n_group=8, topk_group=4, group_top=2, scale=2.5,
                                scores=scores, out=out, workspace=ws)
    assert got is out and s is scores
    whole = m.Routing(*[getattr(out, f) for f in ("topk_ids", "topk_w", "counts", "offsets", "perm_src_token", "perm_of_assignment")],
                      out.perm_weight if weights else _call(t, c, bias).perm_weight)
    _check(whole, scores, _want(l, c, bias), k, E)
    for w, n in guard:
        assert (w[:5] == 77).all() and (w[5 + n:] == 77).all()
