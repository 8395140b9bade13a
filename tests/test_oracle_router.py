"""The float64 references of the router, the combine's gradients and INT4: their
gradients against differences, their codes against the definition."""
import numpy as np
import pytest

from oracle import int4 as Q
from oracle import moe as OM
from oracle import router as R


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(kind, renormalize):
    r = np.random.default_rng([3, renormalize])
    T, E, k, h = 5, 9, 3, 1e-6
    l, dw, ds = r.standard_normal((T, E)), r.standard_normal((T, k)), r.standard_normal((T, E))
    bias = r.standard_normal(E) * 0.1
    ids, _, _, is_open = R.route(l, k, kind, bias, renormalize=renormalize, scale=2.5)

    def loss(x):
        return (R.weights(x, ids, is_open, kind, renormalize, 2.5) * dw).sum() + (R.scores(x, kind)[0] * ds).sum()

    got, _ = R.route_grad(dw, l, ids, is_open, kind, renormalize, 2.5, ds)
    for t in range(T):
        for e in range(E):
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: h^2 of a third derivative below 50, and rounding 1e-15 / h
            assert abs((loss(up) - loss(dn)) / (2 * h) - got[t, e]) < 1e-8


def test_combine_gradient_against_differences():
    r = np.random.default_rng(4)
    T, k, H = 3, 2, 8
    dout, y, w = r.standard_normal((T, H)), r.standard_normal((T * k, H)), r.random((T, k))
    rows = r.permutation(T * k).reshape(T, k)
    (dy, _), (dw, _) = R.combine_grad(dout, y, rows, w)

    def loss(y, w):
        return sum((w[t, j] * y[rows[t, j]] * dout[t]).sum() for t in range(T) for j in range(k))

    for a, grad in ((y, dy), (w, dw)):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += 0.5
            dn[i] -= 0.5
            # linear: the difference is the gradient
            diff = loss(up, w) - loss(dn, w) if a is y else loss(y, up) - loss(y, dn)
            assert abs(diff - grad[i]) < 1e-12


def test_plain_softmax_router_is_the_older_one():
    l = np.random.default_rng(5).standard_normal((20, 12)).astype(np.float32)
    ids, w, _, _ = R.route(l, 4)
    want_ids, want_w = OM.route(l, 4)
    assert np.array_equal(ids, want_ids) and np.allclose(w, want_w, rtol=2.0 ** -23, atol=0)


def test_closed_experts_and_groups():
    n, i = np.nan, np.inf
    l = np.array([[n, -i, 1, 0, 3, 3, -i, -i], [-i] * 8, [0, 5, 1, 1, 1, 1, -i, 2]])
    ids, w, s, _ = R.route(l, 3, "sigmoid", n_group=4, topk_group=2, group_top=2)
    assert ids[0].tolist() == [4, 5, 2] and ids[1].tolist() == [0, 1, 2] and ids[2].tolist() == [1, 2, 3]
    assert (w[1] == 0).all() and np.allclose(w.sum(1), [1, 0, 1]) and s[0, 0] == 0
    # one open expert in a group counts alone; three wanted, two open: the rest by id with weight 0
    ids, w, _, _ = R.route(np.array([[-i, 4.0, -i, -i, 1.0, -i]]), 3, n_group=2, topk_group=2, group_top=2)
    assert ids[0].tolist() == [1, 4, 0] and w[0, 2] == 0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_int4_values_are_within_half_a_step(zeros, dtype):
    r = np.random.default_rng(6)
    x = r.standard_normal((7, 256)).astype(np.float32)
    codes, s, z = Q.quantize(x, 64, zeros, dtype)
    v = Q.dequantize(codes, s, z, 64)
    step = np.repeat(s, 64, -1).astype(np.float64)
    # half a step, half more where the zero point's rounding moves an end, and the
    # scale's own rounding (relative eps / 2, times 15 steps)
    bound = step * ((1.0 if zeros else 0.5) + 15 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -11) + 1e-5)
    assert (np.abs(v - x) <= bound).all()


def test_int4_edges():
    x = np.zeros((4, 64), np.float32)
    x[1, 0], x[2, 40], x[3, :32] = np.nan, np.inf, 3.0
    for zeros, empty in ((False, 8), (True, 0)):
        codes, s, z = Q.quantize(x, 32, zeros, "f16")
        assert np.isnan(s[1, 0]) and s[1, 1] == 1 and np.isnan(s[2, 1]) and (codes[0] == empty * 17).all()
        assert (codes[1, :16] == empty * 17).all()
        assert z is None or (z[0] == 0).all()
    assert np.isnan(Q.quantize(np.full((1, 32), 1e6, np.float32), 32, False, "f16")[1]).all()     # the scale overflows
