"""A training step of MoELayer16 (routing, both products, all gradients, memory
of its own for each) and gradients summed in parts, captured once and replayed
between eager steps with new contents: the same bytes every time."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import MoELayer16
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu


def _normal(r, shape, std=1.0):
    return torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16).to(DEV)


def _replay(step, refresh):
    """step() eagerly, captured, and replayed with other inputs between eager steps."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        refresh()
        graph.replay()
        torch.cuda.synchronize()
        copy = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(copy, want)):
            assert torch.equal(a, b), (i, n)


def test_a_layers_training_step():
    r = np.random.default_rng(71)
    T, H, I, E, k = 120, 264, 136, 7, 3
    logits, x, dy = torch.randn((T, E), device=DEV), _normal(r, (T, H)), _normal(r, (T * k, H))
    w_gu, w_dn = _normal(r, (E, 2 * I, H), 0.06), _normal(r, (E, H, I), 0.08)
    layer = MoELayer16(T, H, I, E, k, DEV)

    def step():
        layer.route(logits)
        gu = torch.empty((T * k, 2 * I), device=DEV)
        y = layer.expert_rows(x, w_gu, w_dn, gu=gu)
        return (y.clone(),) + layer.expert_rows_backward(dy, gu, x, w_gu, w_dn)

    def refresh():
        logits.copy_(torch.randn((T, E), device=DEV))
        for t in (x, dy):
            t.copy_(_normal(r, t.shape))

    _replay(step, refresh)


def test_gradients_in_parts_and_int8():
    r = np.random.default_rng(72)
    M, N, K = 1100, 1032, 72
    a, b, dy = _normal(r, (M, K)), _normal(r, (1, N, K), 0.1), _normal(r, (M, N))
    off = torch.tensor([0, M - 5], dtype=torch.int32, device=DEV)
    assert m.lib().moe_grouped_gemm_backward_workspace_size(1, N, K, M) > 0
    # int8 needs multiples of 16
    x, w = _normal(r, (M, 80)), m.int8_quantize(_normal(r, (1, N, 80)))

    def step():
        da = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
        db = m.moe_grouped_gemm_backward(dy, a, b, off, da=da)[1]
        q = m.int8_quantize(x)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
        m.int8_grouped_gemm(q, w, off, m_total=M, out=y)
        return da, db, q.codes, q.scales, y

    def refresh():
        for t in (a, dy, x):
            t.copy_(_normal(r, t.shape))

    _replay(step, refresh)


def test_a_captured_fork_whose_calls_allocate():
    """Calls on a second stream of the capture, with memory of their own, beside one on the first."""
    r = np.random.default_rng(73)
    M, H, I, E = 500, 136, 264, 3
    x, w, dh = _normal(r, (M, H)), _normal(r, (E, 2 * I, H), 0.1), _normal(r, (M, I))
    off = torch.tensor([0, 200, 201, M], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        h, gu = m.moe_gated_ffn(x, w, off, m_total=M, save_gu=True, stream=side)
        dx, dw = m.moe_gated_ffn_backward(dh, gu, x, w, off, stream=side)
        q = m.int8_quantize(x)
        here.wait_stream(side)
        return h, dx, dw, q.codes, q.scales

    def refresh():
        for t in (x, dh):
            t.copy_(_normal(r, t.shape))

    _replay(step, refresh)
