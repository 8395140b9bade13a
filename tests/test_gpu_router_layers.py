"""Layers with a Router, the INT4 layer and the 16-bit layer's whole training step:
the calls together as they are used, on streams and in captured graphs."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import (FP8MoELayer, INT4MoELayer, INT8MoELayer, MoELayer, MoELayer16, MXMoELayer, Router,
                                                quantize_expert_weights, quantize_expert_weights_fp8, quantize_expert_weights_int4,
                                                quantize_expert_weights_int8, quantize_expert_weights_mx)
from oracle import int4 as Q
from oracle import router as R
from tests.gpu_common import DEV
from tests.test_gpu_experts_graphs import _replay

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _normal(shape, std=1.0, dtype=BF):
    return (torch.randn(shape, device=DEV) * std).to(dtype)


def _router(E, bias=True):
    return Router(m.SCORE_SIGMOID, torch.randn(E, device=DEV) * 0.1 if bias else None, n_group=4, topk_group=2, group_top=2, scale=2.5)


@pytest.mark.parametrize("T", [3, 200, 700])
def test_int4_layer(T):
    """Both paths (4-bit kernels, dequantised weights) against the layer's steps in float64."""
    H, I, E, k = 256, 128, 8, 2
    logits, x = torch.randn((T, E), device=DEV), _normal((T, H))
    w_gu, w_dn = _normal((E, 2 * I, H), 0.06), _normal((E, H, I), 0.08)
    w = quantize_expert_weights_int4(w_gu, w_dn, 64, T % 2 == 1)
    router = _router(E)
    layer = INT4MoELayer(T, H, I, E, k, DEV, router)
    assert layer.wide == (T * k > layer.most_rows * E)
    out = layer.forward(logits, x, w).double().cpu().numpy()
    ids, wt, _, _ = R.route(logits.cpu().numpy(), k, "sigmoid", router.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
    vals = [Q.dequantize(q.codes.cpu().numpy(), q.scales.float().cpu().numpy(), None if q.zeros is None else q.zeros.cpu().numpy(), 64)
            for q in (w.gu, w.dn)]
    xs = x.double().cpu().numpy()
    for t in range(T):
        want, size = np.zeros(H), np.zeros(H)
        for j in range(k):
            e = ids[t, j]
            y = vals[0][e] @ xs[t]
            h = y[:I] / (1 + np.exp(-y[:I])) * y[I:]
            row = vals[1][e] @ h
            want += wt[t, j] * row
            # roundings to bf16: the weights (where they are dequantised), y's effect in h, h, the row; then the sum
            size += wt[t, j] * (np.abs(vals[1][e]) @ (np.abs(h) + 1.13 * (np.abs(vals[0][e][:I]) @ np.abs(xs[t])) * np.abs(y[I:])
                                                      + np.abs(y[:I]) * (np.abs(vals[0][e][I:]) @ np.abs(xs[t]))) + np.abs(row))
        assert (np.abs(out[t] - want) <= 2.0 ** -8 * (2 * size + np.abs(want)) + 1e-6).all()


@pytest.mark.parametrize("kind", ["nvfp4", "mx", "fp8", "int8", "16"])
def test_layers_take_a_router(kind):
    """A layer with a Router gives what its own steps give on that routing: here, against the plain
    softmax layer on logits whose softmax router makes the same choices and weights."""
    T, H, I, E, k = 20, 256, 128, 8, 2
    logits, x = torch.randn((T, E), device=DEV), _normal((T, H))
    w_gu, w_dn = _normal((E, 2 * I, H), 0.06), _normal((E, H, I), 0.08)
    router = Router(m.SCORE_SIGMOID, renormalize=True)
    r = m.moe_route_scored(logits, k, score=m.SCORE_SIGMOID)
    same = torch.full((T, E), -60.0, device=DEV).scatter_(1, r.topk_ids.long(), r.topk_w.double().log().float())
    if kind == "nvfp4":
        w, g = quantize_expert_weights(w_gu, w_dn).pack(), torch.tensor([1e-3], device=DEV)
        make, run = MoELayer, lambda l, lg: l.forward(lg, x, w, g)
    elif kind == "16":
        make, run = MoELayer16, lambda l, lg: l.forward(lg, x, w_gu, w_dn)
    else:
        make, quant = {"mx": (MXMoELayer, quantize_expert_weights_mx), "fp8": (FP8MoELayer, quantize_expert_weights_fp8),
                       "int8": (INT8MoELayer, quantize_expert_weights_int8)}[kind]
        w = quant(w_gu, w_dn)
        run = lambda l, lg: l.forward(lg, x, w)  # noqa: E731
    a, b = make(T, H, I, E, k, DEV, router=router), make(T, H, I, E, k, DEV)
    got, want = run(a, logits).clone(), run(b, same).clone()
    assert torch.equal(a.routing.topk_ids, b.routing.topk_ids) and torch.equal(a.routing.offsets, b.routing.offsets)
    # the two weights differ by a few float32 steps (a logarithm and back: |log w| + 4 of them),
    # which moves a bf16 result by at most its last place beyond that
    tol = 2.0 ** -7 * want.float().abs() + 2.0 ** -18 * want.float().abs().max()
    assert ((got.float() - want.float()).abs() <= tol).all()


def test_training_step_against_differences():
    """dlogits, dx and the weights' gradients of the 16-bit layer against central differences of a
    float64 evaluation on the same choices, at a few places each."""
    torch.manual_seed(3)
    T, H, I, E, k = 24, 128, 64, 8, 2
    logits, x = torch.randn((T, E), device=DEV), _normal((T, H))
    w_gu, w_dn = _normal((E, 2 * I, H), 0.09), _normal((E, H, I), 0.12)
    dout, ds = _normal((T, H)), torch.randn(E, device=DEV) * 0.1
    router = _router(E)
    layer = MoELayer16(T, H, I, E, k, DEV, router=router)
    gu = torch.empty((T * k, 2 * I), device=DEV)
    layer.forward(logits, x, w_gu, w_dn, gu=gu)
    grads = [g.double().cpu().numpy() for g in layer.backward(dout, gu, logits, x, w_gu, w_dn, d_scores=ds)]
    ids = layer.routing.topk_ids.cpu().numpy()
    args = [t.double().cpu().numpy() for t in (logits, x, w_gu, w_dn)]
    dn, dsn = dout.double().cpu().numpy(), ds.double().cpu().numpy()

    def loss(a):
        lg, xs, gu_w, dn_w = a
        wt = R.weights(lg, ids, np.ones((T, E), bool), "sigmoid", True, 2.5)
        total = (R.scores(lg, "sigmoid")[0] * dsn).sum()
        for t in range(T):
            for j in range(k):
                y = gu_w[ids[t, j]] @ xs[t]
                total += wt[t, j] * (dn_w[ids[t, j]] @ (y[:I] / (1 + np.exp(-y[:I])) * y[I:])) @ dn[t]
        return total

    r, h = np.random.default_rng(4), 1e-5
    for i, g in enumerate(grads):
        big = np.sqrt((g ** 2).mean())
        for _ in range(6):
            at = tuple(r.integers(0, n) for n in g.shape)
            moved = []
            for step in (h, -h):
                a = [v.copy() if n == i else v for n, v in enumerate(args)]
                a[i][at] += step
                moved.append(loss(a))
            diff = (moved[0] - moved[1]) / (2 * h)
            # three bf16 roundings on the way (h, dy, pre-activation gradients) and the result's, on sums
            # of at most 2 k H terms of the gradient's typical size: 4 * 2^-8 of that and of the value
            assert abs(g[at] - diff) <= 2.0 ** -6 * (abs(diff) + 2 * big), (i, at, g[at], diff)


def test_gradients_of_another_call_are_refused():
    T, H, I, E, k = 8, 64, 32, 4, 2
    layer = MoELayer16(T, H, I, E, k, DEV)
    ops = (torch.randn((T, E), device=DEV), _normal((T, H)), _normal((E, 2 * I, H)), _normal((E, H, I)))
    gu, dout = torch.empty((T * k, 2 * I), device=DEV), _normal((T, H))
    layer.forward(*ops, gu=gu)
    assert len(layer.backward(dout, gu, *ops)) == 4
    layer.forward(*ops)
    with pytest.raises(ValueError, match="forward"):
        layer.backward(dout, gu, *ops)


@pytest.mark.parametrize("T", [2, 120])
def test_captured_int4_step(T):
    H, I, E, k = 256, 64, 8, 2
    logits, x = torch.randn((T, E), device=DEV), _normal((T, H))
    w = quantize_expert_weights_int4(_normal((E, 2 * I, H), 0.06), _normal((E, H, I), 0.08), 64)
    layer = INT4MoELayer(T, H, I, E, k, DEV, _router(E))

    def step():
        out = layer.forward(logits, x, w)
        return (out.clone(),) + tuple(t.clone() for t in vars(layer.routing).values())

    def refresh():
        logits.copy_(torch.randn((T, E), device=DEV))
        x.copy_(_normal((T, H)))

    _replay(step, refresh)


@pytest.mark.parametrize("T", [120, 2100])
def test_captured_training_step(T):
    H, I, E, k = 264, 136, 12, 3
    logits, x, dout = torch.randn((T, E), device=DEV), _normal((T, H)), _normal((T, H))
    w_gu, w_dn = _normal((E, 2 * I, H), 0.06), _normal((E, H, I), 0.08)
    layer = MoELayer16(T, H, I, E, k, DEV, router=_router(E))
    ds = torch.randn(E, device=DEV)

    def step():
        gu = torch.empty((T * k, 2 * I), device=DEV)
        out = layer.forward(logits, x, w_gu, w_dn, gu=gu)
        return (out.clone(),) + layer.backward(dout, gu, logits, x, w_gu, w_dn, d_scores=ds)

    def refresh():
        logits.copy_(torch.randn((T, E), device=DEV))
        for t in (x, dout):
            t.copy_(_normal(t.shape))

    _replay(step, refresh)


def test_captured_weights_on_two_streams():
    """Quantising, its inverse and a product on a second stream of a capture, beside a routing on the first."""
    T, E, K, N = 30, 16, 256, 80
    logits, w, x = torch.randn((T, E), device=DEV), torch.randn((1, N, K), device=DEV), _normal((T, K))
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        q = m.int4_quantize(w, 64, True, stream=side)
        v = m.int4_dequantize(q, stream=side)
        y = m.int4_grouped_gemv(x, q, off, m_total=T, stream=side)
        r = m.moe_route_scored(logits, 4, score=m.SCORE_SIGMOID)
        here.wait_stream(side)
        return q.codes, q.scales.view(torch.int16), q.zeros, v, y, r.topk_ids, r.topk_w, r.perm_src_token

    def refresh():
        for t in (logits, w):
            t.copy_(torch.randn(t.shape, device=DEV))
        x.copy_(_normal(x.shape))

    _replay(step, refresh)


def test_two_streams_at_once():
    """The same calls on two streams side by side, each with memory of its own, give the bytes of one after the other."""
    T, E, k, H, I = 2300, 64, 4, 256, 64
    sets = []
    for i in range(2):
        torch.manual_seed(i)
        sets.append((torch.randn((T, E), device=DEV), torch.randn(E, device=DEV) * 0.1, _normal((T, H)),
                     m.int4_quantize(torch.randn((E, 2 * I, H), device=DEV) * 0.1, 64)))

    def work(s, stream):
        logits, bias, x, b = s
        r = m.moe_route_scored(logits, k, score=m.SCORE_SIGMOID, bias=bias, n_group=8, topk_group=3, group_top=2, stream=stream)
        h = m.int4_grouped_gemv(x, b, r.offsets, m_total=T * k, a_rows=r.perm_src_token, gated=True, stream=stream)
        dy, dw = m.moe_unpermute_combine_backward(x[:, :I].contiguous(), h, r.perm_of_assignment, r.topk_w, stream=stream)
        d = m.moe_route_scored_backward(dw, logits, r.topk_ids, score=m.SCORE_SIGMOID, stream=stream)
        return (r.topk_ids, r.topk_w, r.perm_src_token, r.perm_of_assignment, h, dy, dw, d)

    want = [work(s, None) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(work(s, None))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_debug_checks(monkeypatch):
    monkeypatch.setenv("NVFP4MOE_DEBUG", "1")
    b = m.int4_quantize(torch.randn((2, 16, 64), device=DEV), 32)
    x = _normal((4, 64))
    with pytest.raises(m.NVFP4MoEError, match="offsets"):
        m.int4_grouped_gemv(x, b, torch.tensor([0, 5, 4], dtype=torch.int32, device=DEV), m_total=4)
    with pytest.raises(m.NVFP4MoEError, match="a_rows"):
        m.int4_grouped_gemv(x, b, torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV), m_total=4,
                            a_rows=torch.tensor([0, 1, 2, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(m.NVFP4MoEError, match="perm_of_assignment"):
        m.moe_unpermute_combine_backward(_normal((2, 64)), x, torch.tensor([0, 1, 2, 4], dtype=torch.int32, device=DEV),
                                         torch.ones((2, 2), device=DEV))
    m.int4_grouped_gemv(x, b, torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV), m_total=4)
