"""The router's scores through the 16-bit layer: a training step with a balance loss on
them, with the calls of the layer alone."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import MoELayer16, Router
from oracle import router as R
from tests.gpu_common import DEV
from tests.test_gpu_experts_graphs import _replay
from tests.test_gpu_router_layers import _normal, _router

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _sizes(T):
    H, I, E, k = 128, 64, 8, 2
    return H, I, E, k, (torch.randn((T, E), device=DEV), _normal((T, H)), _normal((E, 2 * I, H), 0.09), _normal((E, H, I), 0.12))


def _balance(layer, s, k):
    """E sum_e f_e mean_t s_te with f the share of the assignments: its gradient, one row for all tokens."""
    T, E = s.shape
    return layer.routing.counts.float() * (E / (T * k * T))


@pytest.mark.parametrize("T", [9, 2100])
@pytest.mark.parametrize("how", ["plain", "softmax", "sigmoid"])
def test_step_with_a_balance_loss(how, T):
    H, I, E, k, ops = _sizes(T)
    router = {"plain": None, "softmax": Router(bias=torch.randn(E, device=DEV) * 0.1, renormalize=False), "sigmoid": _router(E)}[how]
    layer, other = (MoELayer16(T, H, I, E, k, DEV, router=router) for _ in range(2))
    s, gu = torch.full((T, E), -1.0, device=DEV), torch.empty((T * k, 2 * I), device=DEV)
    out = layer.forward(*ops, gu=gu, scores=s)
    kind = "sigmoid" if how == "sigmoid" else "softmax"
    want = R.scores(ops[0].cpu().numpy(), kind)[0]
    assert (np.abs(s.double().cpu().numpy() - want) <= want * U * (1 + 2.0 ** -15)).all()
    # the same choice as without, and the same step (weights of the plain router to a few of their own roundings)
    gu2 = torch.empty_like(gu)
    out2 = other.forward(*ops, gu=gu2)
    assert torch.equal(layer.routing.topk_ids, other.routing.topk_ids) and torch.equal(gu, gu2)
    if how == "plain":
        assert ((layer.routing.topk_w - other.routing.topk_w).abs() <= 16 * U).all()
    else:
        assert torch.equal(out, out2)
    dout, ds = _normal((T, H)), _balance(layer, s, k)
    got = layer.backward(dout, gu, *ops, d_scores=ds)
    none = layer.backward(dout, gu, *ops)
    # the balance loss adds its own gradient to the logits' alone
    for a, b in zip(got[1:], none[1:]):
        assert torch.equal(a, b)
    l = ops[0].cpu().numpy()
    zero = np.zeros((T, k), np.float32)
    ids = layer.routing.topk_ids.cpu().numpy()
    d, tol = R.route_grad(zero, l, ids, np.ones((T, E), bool), kind, True, 1.0, ds.cpu().numpy())
    added = got[0].double().cpu().numpy() - none[0].double().cpu().numpy()
    # both gradients are float32 results of the same chain: their difference has the rounding of each, of terms
    # of the scores' part and of the weights' (below 32 half steps of what the two sum up from)
    size = np.abs(none[0].double().cpu().numpy()) + np.abs(got[0].double().cpu().numpy())
    big = size.max(1, keepdims=True) + np.abs(d).max()
    assert (np.abs(added - d) <= tol + 64 * U * big).all()


def test_captured_step_with_scores():
    T = 120
    H, I, E, k, ops = _sizes(T)
    layer = MoELayer16(T, H, I, E, k, DEV, router=_router(E))
    dout = _normal((T, H))

    def step():
        gu, s = torch.empty((T * k, 2 * I), device=DEV), torch.empty((T, E), device=DEV)
        out = layer.forward(*ops, gu=gu, scores=s)
        return (out.clone(), s) + layer.backward(dout, gu, *ops, d_scores=_balance(layer, s, k))

    def refresh():
        ops[0].copy_(torch.randn((T, E), device=DEV))
        ops[1].copy_(_normal((T, H)))

    _replay(step, refresh)


def test_scores_of_another_shape_are_refused():
    T = 9
    H, I, E, k, ops = _sizes(T)
    layer = MoELayer16(T, H, I, E, k, DEV)
    for s in (torch.empty((T, E + 1), device=DEV), torch.empty((T, E), dtype=torch.bfloat16, device=DEV)):
        with pytest.raises((ValueError, TypeError)):
            layer.forward(*ops, scores=s)
