"""The router's reference where a bias closes an expert: values written out by hand."""
import numpy as np
import pytest

from oracle import router as R


@pytest.mark.parametrize("closed", [-np.inf, np.nan])
def test_bias_closes_the_choice_alone(closed):
    l, bias = np.zeros((1, 4)), np.array([0, closed, 0.5, 0])
    ids, w, s, is_open = R.route(l, 4, "softmax", bias, renormalize=False, scale=2.0)
    assert ids[0].tolist() == [2, 0, 3, 1] and w[0].tolist() == [0.5, 0.5, 0.5, 0] and s[0].tolist() == [0.25] * 4
    d, _ = R.route_grad(np.zeros((1, 2)), l, ids[:, :2], is_open, "softmax", False, 1.0, np.array([0, 1.0, 0, 0]))
    assert (d[0] * 16).tolist() == [-1, 3, -1, -1]
    ids, w, s, is_open = R.route(l, 4, "sigmoid", bias, renormalize=False)
    assert ids[0].tolist() == [2, 0, 3, 1] and w[0].tolist() == [0.5, 0.5, 0.5, 0] and s[0].tolist() == [0.5] * 4
    d, _ = R.route_grad(np.array([[0, 0, 0, 1.0]]), l, ids, is_open, "sigmoid", False, 1.0, np.array([0, 1.0, 0, 0]))
    assert d[0].tolist() == [0, 0.25, 0, 0]
