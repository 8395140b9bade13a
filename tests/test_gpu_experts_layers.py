"""The INT8 layer and the 16-bit layer as a user runs them: every stage in
order on one routing, each checked against the oracle from the GPU's own inputs
of that stage (bit for bit where the stage is exact), the experts' gradients
through both products, and a captured layer step."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import INT8MoELayer, MoELayer16, quantize_expert_weights_int8
from oracle import experts16 as X
from oracle import int8 as Q
from oracle import moe as OM
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu
T, H, I, E, K = 70, 256, 128, 8, 3


def _inputs(seed):
    r = np.random.default_rng(seed)
    logits = r.standard_normal((T, E)).astype(np.float32)
    logits[:, 5] = -30 - np.arange(T)              # an expert without rows
    x = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w_gu = torch.from_numpy((r.standard_normal((E, 2 * I, H)) / 16).astype(np.float32)).to(torch.bfloat16)
    w_dn = torch.from_numpy((r.standard_normal((E, H, I)) / 12).astype(np.float32)).to(torch.bfloat16)
    return r, up(logits), x.to(DEV), w_gu.to(DEV), w_dn.to(DEV)


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, tol, what):
    err = np.abs(_f64(got) - want)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.3f} of the bound"


def _combine(y, r, tol_y=0.0):
    """The combine in float64 of float32-weighted rows and its bound (k float32 fused steps, one bf16 rounding)."""
    perm, w = r.perm_of_assignment.cpu().numpy(), _f64(r.topk_w)
    rows = y[perm].reshape(T, K, -1)
    out = np.einsum("tj,tjh->th", w, rows)
    mag = np.einsum("tj,tjh->th", np.abs(w), np.abs(rows))
    return out, (K + 1) * X.U * mag * 1.01 + X.HALF["bf16"] * np.abs(out) + X.TINY["bf16"]


def test_int8_layer_stage_by_stage():
    _, logits, x, w_gu, w_dn = _inputs(1)
    w = quantize_expert_weights_int8(w_gu, w_dn)
    layer = INT8MoELayer(T, H, I, E, K, DEV)
    out = layer.forward(logits, x, w)
    r = layer.routing
    ids, _ = OM.route(logits.cpu().numpy(), K)
    _, off, src, _, _ = OM.permute(ids, np.zeros((T, K), np.float32), E)
    assert np.array_equal(r.offsets.cpu().numpy(), off) and np.array_equal(r.perm_src_token.cpu().numpy(), src)
    codes = {}
    for name, t, q in (("x", x, layer.xq), ("gu", w_gu, w.gu), ("dn", w_dn, w.dn), ("h", layer.h, layer.hq)):
        c, s = Q.quantize(t.float().cpu().numpy())
        assert np.array_equal(q.codes.cpu().numpy(), c) and np.array_equal(q.scales.cpu().numpy(), s), name
        codes[name] = (c, s)
    y, tol = Q.grouped_gemm(*codes["x"], *codes["gu"], off, src)
    h, th = Q.swiglu(y, tol)
    _close(layer.h, h, Q.rounded(h, th, "bf16"), "h")
    y, tol = Q.grouped_gemm(*codes["h"], *codes["dn"], off)
    _close(layer.y2, y, Q.rounded(y, tol, "bf16"), "y")
    _close(out, *_combine(_f64(layer.y2), r), "out")


def test_int8_layer_step_in_a_graph():
    r, logits, x, w_gu, w_dn = _inputs(2)
    w = quantize_expert_weights_int8(w_gu, w_dn)
    a, b = INT8MoELayer(T, H, I, E, K, DEV), INT8MoELayer(T, H, I, E, K, DEV)
    a.forward(logits, x, w)
    b.forward(logits, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(logits, x, w)
    for i in range(4):
        logits.copy_(up(r.standard_normal((T, E)).astype(np.float32)))
        x.copy_(torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16))
        b.out.zero_()
        graph.replay()
        want = a.forward(logits, x, w)
        torch.cuda.synchronize()
        assert torch.equal(want, b.out), i


@pytest.mark.parametrize("activation,kind", [(m.ACT_SILU, "silu"), (m.ACT_GELU, "gelu")])
def test_layer16_forward_and_expert_gradients(activation, kind):
    rng, logits, x, w_gu, w_dn = _inputs(3)
    layer = MoELayer16(T, H, I, E, K, DEV, activation=activation)
    out = layer.forward(logits, x, w_gu, w_dn)
    r = layer.routing
    off, src = r.offsets.cpu().numpy(), r.perm_src_token.cpu().numpy()
    x64, gu64, dn64 = _f64(x), _f64(w_gu), _f64(w_dn)
    (h, th), _ = X.gated(x64, gu64, off, src, kind)
    _close(layer.h, h, th, "h")
    _close(layer.y2, *X.product(_f64(layer.h), dn64, off), "y")
    _close(out, *_combine(_f64(layer.y2), r), "out")

    gu = torch.empty((T * K, 2 * I), device=DEV)
    y = layer.expert_rows(x, w_gu, w_dn, gu=gu).clone()
    dy = torch.from_numpy(rng.standard_normal((T * K, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dx, dw_gu, dw_dn = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn)
    assert torch.equal(y, layer.y2)
    h64 = _f64(layer.h)
    (dh, tdh), (rdn, tdn) = X.product_grad(_f64(dy), h64, dn64, off)
    _close(dw_dn, rdn, tdn, "dw_dn")
    # the gated block's gradients from the GPU's own (bf16) dh
    dh_gpu, _ = m.moe_grouped_gemm_backward(dy, layer.h, w_dn, r.offsets, need_db=False)
    _close(dh_gpu, dh, tdh, "dh")
    (rows, trows), (rgu, tgu) = X.gated_grad(_f64(dh_gpu), x64, gu64, off, src, kind)
    _close(dw_gu, rgu, tgu, "dw_gu")
    # a token's gradient: the sum of its k rows (each within its bound), k float32 additions, one rounding
    perm = r.perm_of_assignment.cpu().numpy()
    want = rows[perm].reshape(T, K, H).sum(1)
    tol = trows[perm].reshape(T, K, H).sum(1)
    mag = np.abs(rows[perm]).reshape(T, K, H).sum(1) + tol
    _close(dx, want, (tol + (K + 1) * X.U * mag) * (1 + X.HALF["bf16"]) + X.HALF["bf16"] * np.abs(want), "dx")
    assert not dw_gu[5].any() and not dw_dn[5].any()


def test_layer16_gradients_on_another_stream():
    """The rows between the two backward calls belong to the call alone; their
    memory is not handed out again before the side stream has read them."""
    rng, logits, x, w_gu, w_dn = _inputs(5)
    layer = MoELayer16(T, H, I, E, K, DEV)
    layer.route(logits)
    gu = torch.empty((T * K, 2 * I), device=DEV)
    layer.expert_rows(x, w_gu, w_dn, gu=gu)
    dy = torch.from_numpy(rng.standard_normal((T * K, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    want = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn((2048, 2048), device=DEV)
    for _ in range(3):
        with torch.cuda.stream(side):
            busy @ busy
        got = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn, stream=side)
        for cols in (I, H):                        # would take the freed rows
            torch.full((T * K, cols), float("nan"), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layer16_float16_rows():
    rng, logits, x, w_gu, w_dn = _inputs(4)
    x, w_gu, w_dn = x.half(), w_gu.half(), w_dn.half()
    layer = MoELayer16(T, H, I, E, K, DEV, dtype=torch.float16)
    r = layer.route(logits)
    gu = torch.empty((T * K, 2 * I), device=DEV)
    layer.expert_rows(x, w_gu, w_dn, gu=gu)
    dy = torch.from_numpy(rng.standard_normal((T * K, H)).astype(np.float32)).half().to(DEV)
    dx, dw_gu, dw_dn = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn)
    off, src = r.offsets.cpu().numpy(), r.perm_src_token.cpu().numpy()
    _close(layer.y2, *X.product(_f64(layer.h), _f64(w_dn), off, None, "f16"), "y")
    _close(dw_dn, *X.product_grad(_f64(dy), _f64(layer.h), _f64(w_dn), off, None, "f16")[1], "dw_dn")
    assert dx.shape == (T * K, H) and torch.isfinite(dx).all() and dw_gu.shape == w_gu.shape
