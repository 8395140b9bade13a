"""Calls on an idle side stream while the current stream still has work queued
that writes memory which it has already freed: the results are those of a call
on the current stream, since the call's own memory is the side stream's."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import MoELayer16
from tests.gpu_common import DEV

pytestmark = pytest.mark.gpu
M, H, I, E = 700, 512, 256, 2


def _operands():
    r = np.random.default_rng(61)

    def t(*shape, std=1.0):
        return torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16).to(DEV)

    x, w = t(M, H), t(E, 2 * I, H, std=0.05)
    off = torch.tensor([0, 300, M], dtype=torch.int32, device=DEV)
    return dict(x=x, w=w, off=off, dh=t(M, I), dy=t(M, 2 * I), gu=t(M, 2 * I).float(), q=m.int8_quantize(x),
                wq=m.int8_quantize(w))


CALLS = {
    "gated": lambda o, s: m.moe_gated_ffn(o["x"], o["w"], o["off"], m_total=M, save_gu=True, stream=s),
    "gated_backward": lambda o, s: m.moe_gated_ffn_backward(o["dh"], o["gu"], o["x"], o["w"], o["off"], stream=s),
    "product": lambda o, s: (m.moe_grouped_gemm(o["x"], o["w"], o["off"], m_total=M, stream=s),),
    "product_backward": lambda o, s: m.moe_grouped_gemm_backward(o["dy"], o["x"], o["w"], o["off"], stream=s),
    "int8_quantize": lambda o, s: (lambda q: (q.codes, q.scales))(m.int8_quantize(o["x"], stream=s)),
    "int8_product": lambda o, s: (m.int8_grouped_gemm(o["q"], o["wq"], o["off"], m_total=M, stream=s),),
    "combine": lambda o, s: (m.moe_unpermute_combine(o["x"], None, None, M // 2, 2, stream=s),),
}


@pytest.mark.parametrize("name", CALLS)
def test_call_beside_pending_work_on_freed_memory(name):
    o = _operands()
    want = CALLS[name](o, None)
    ws = {"gated_backward": m.lib().moe_gated_ffn_backward_workspace_size(E, H, I, M),
          "product_backward": m.lib().moe_grouped_gemm_backward_workspace_size(E, 2 * I, H, M)}.get(name, 0)
    sizes = [t.numel() * t.element_size() for t in want] + [max(ws, 256)]
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device=DEV)
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        for _ in range(4):
            busy @ busy                       # milliseconds
        for b in blocks:
            b.fill_(255)                      # behind them, into blocks that are free by then
        del b, blocks
        got = CALLS[name](o, side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del a, b, got


def test_layer_gradients_beside_pending_work():
    """dh, the rows' gradients, both workspaces and the token gradient of
    expert_rows_backward are the side stream's, and the last is held for the
    caller's stream."""
    T = 128
    o = _operands()
    x, w_gu = o["x"][:T].contiguous(), o["w"]
    w_dn = o["w"].transpose(1, 2).contiguous()[:, :, :I].contiguous()
    layer = MoELayer16(T, H, I, E, 2, DEV)
    layer.route(o["gu"][:T, :E].contiguous())
    gu = torch.empty((2 * T, 2 * I), device=DEV)
    layer.expert_rows(x, w_gu, w_dn, gu=gu)
    dy = o["x"][T:3 * T].contiguous()
    want = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn)
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device=DEV)
    rows = 2 * T
    sizes = [rows * I * 2, rows * H * 2, T * H * 2, E * 2 * I * H * 2, E * H * I * 2,
             m.lib().moe_gated_ffn_backward_workspace_size(E, H, I, rows),
             max(256, m.lib().moe_grouped_gemm_backward_workspace_size(E, H, I, rows))]
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        for _ in range(4):
            busy @ busy
        for b in blocks:
            b.fill_(255)
        del b, blocks
        got = layer.expert_rows_backward(dy, gu, x, w_gu, w_dn, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        # read on the current stream behind pending work, dropped before that has run, and its memory asked for again
        torch.cuda.current_stream().wait_stream(side)
        busy @ busy
        copy = got[0].clone()
        del a, b, got
        with torch.cuda.stream(side):
            torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(copy, want[0])


def test_block_scaled_calls_beside_pending_work():
    """The same of the calls on block-scaled operands: operands quantised, and
    multiplied, on the side stream."""
    o = _operands()

    def calls(s):
        a, b = m.nvfp4_quantize(o["x"], stream=s), m.mxfp4_quantize(o["x"], stream=s)
        w = m.nvfp4_quantize(o["w"].view(-1, H), stream=s)
        codes, scales = w.codes.view(E, 2 * I, H // 2), w.scales.view(E, 2 * I, H // 16)
        g = _two(w.g, s)
        y = m.nvfp4_grouped_gemm(a, codes, scales, g, o["off"], m_total=M, stream=s)
        q = m.moe_swiglu(y, stream=s)
        mw = m.mxfp4_quantize(o["w"], stream=s)
        z = m.mxfp4_grouped_gemm(b, mw, o["off"], m_total=M, stream=s)
        f = m.fp8_quantize(o["x"], stream=s)
        r = m.moe_route_permute(logits, 8, stream=s)
        return (a.codes, a.scales, b.codes, y, q.codes, q.scales, z, f.codes, f.scales, r.topk_ids, r.perm_src_token)

    def _two(t, s):
        with torch.cuda.stream(s):
            return t.expand(E).contiguous()

    logits = o["gu"][:, :64].contiguous()
    want = calls(None)
    sizes = [t.numel() * t.element_size() for t in want] * 2
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device=DEV)
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        for _ in range(4):
            busy @ busy
        for b in blocks:
            b.fill_(255)
        del b, blocks
        got = calls(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del a, b, got
