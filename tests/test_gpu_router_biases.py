"""Groups chosen by keys of large finite biases: two keys of a group that cancel leave
a value far smaller than the rounding of either, so float32 keys order groups wrongly
where float64 ones do not.  Ids exactly as oracle/router.py has them."""
import numpy as np
import pytest

import block_scaled_fp4_permute_amd as m
from tests.gpu_common import up
from tests.test_gpu_router import KIND
from tests.test_gpu_router_borders import _same

pytestmark = pytest.mark.gpu


def _sigmoid(x):
    return 1 / (1 + np.exp(-x.astype(np.float64)))


def _near_groups(T, E, n, B, seed):
    """Rows whose groups' two largest keys are +B and -B plus scores, the groups' sums of scores a few
    steps of B's rounding apart; the other experts' biases are lower still."""
    r = np.random.default_rng([T, E, n, seed])
    size = E // n
    bias = np.full((n, size), -3.0 * B, np.float32) + r.standard_normal((n, size)).astype(np.float32)
    at = np.argsort(r.random((n, size)), 1)[:, :2]
    g = np.arange(n)
    bias[g, at[:, 0]], bias[g, at[:, 1]] = B, -B
    l = r.standard_normal((T, n, size)).astype(np.float32)
    total = _sigmoid(l[:, 0, at[0, 0]]) + _sigmoid(l[:, 0, at[0, 1]])
    for i in range(1, n):
        first = np.clip(total / 2 + r.uniform(-0.05, 0.05, T), 0.02, 0.98)
        l[:, i, at[i, 0]] = np.log(first / (1 - first))
        rest = total - _sigmoid(l[:, i, at[i, 0]]) + r.uniform(-1, 1, T) * B * 2.0 ** -24
        rest = np.clip(rest, 0.02, 0.98)
        l[:, i, at[i, 1]] = np.log(rest / (1 - rest))
    return l.reshape(T, E), bias.reshape(-1)


def _call(l, k, kind, bias, groups):
    return m.moe_route_scored(up(l), k, score=KIND[kind], bias=up(bias), n_group=groups[0], topk_group=groups[1], group_top=groups[2])


# experts, groups: ends between lanes (64 and 16 a token) and groups of 2, 10 and 12 by way of LDS
SHAPES = [(256, (8, 4, 2)), (64, (2, 1, 2)), (64, (32, 9, 2)), (60, (6, 2, 2)), (72, (6, 3, 2)), (512, (16, 5, 2)), (1000, (8, 3, 2))]


@pytest.mark.parametrize("B", [16.0, 1e3, 1e6])
@pytest.mark.parametrize("T", [16, 2100])
@pytest.mark.parametrize("E,groups", SHAPES, ids=str)
def test_keys_that_cancel_in_a_group(E, groups, T, B):
    print("cancel", E, groups, T, B, flush=True)
    l, bias = _near_groups(T, E, groups[0], B, int(B))
    k = min(8, 2 * groups[1])
    got = _call(l, k, "sigmoid", bias, groups)
    _same(got, l.astype(np.float64), k, "sigmoid", bias, groups, E)


def test_two_groups_of_two():
    """Sums of 16 + s and -16 + s': group 0's are larger in float32, group 1's by 2.5e-7 in float64."""
    l = np.array([[-0.35004669, -0.43241960, 0.60928750, -1.66462743]], np.float32)
    bias = np.array([16, -16, 16, -16], np.float32)
    for T in (1, 40, 2100):
        got = _call(np.tile(l, (T, 1)), 1, "sigmoid", bias, (2, 1, 2))
        assert (got.topk_ids == 2).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [10.0, 1e6, 3e38])
@pytest.mark.parametrize("T", [16, 2100])
@pytest.mark.parametrize("E,groups", SHAPES, ids=str)
def test_large_biases_of_mixed_sign(E, groups, T, B, kind):
    """Random logits; up to 3e38, where a group's sum leaves float32's range and two of them cancel."""
    r = np.random.default_rng([E, T])
    l = r.standard_normal((T, E)).astype(np.float32)
    bias = (r.integers(-1, 2, E) * np.float32(B)).astype(np.float32)
    k = min(8, E // groups[0])
    got = _call(l, k, kind, bias, groups)
    _same(got, l.astype(np.float64), k, kind, bias, groups, E)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T", [16, 2100])
def test_finite_masks(T, top, kind):
    """Experts and whole groups masked by -1e9: those that are left are ordered as without the mask, and
    masked groups by id where too few others are there."""
    E, n = 64, 8
    r = np.random.default_rng(T)
    l = r.standard_normal((T, E)).astype(np.float32)
    for masked in ([5], range(8, 24), range(0, 48), [8 * g + 1 + i for g in range(8) for i in range(7)]):
        bias = np.zeros(E, np.float32)
        bias[list(masked)] = -1e9
        for keep in (2, 5):
            got = _call(l, 8, kind, bias, (n, keep, top))
            _same(got, l.astype(np.float64), 8, kind, bias, (n, keep, top), E)
