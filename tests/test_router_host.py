"""Host-side checks of the router with scores, the combine's gradients and INT4
(no GPU needed): every call below has to be refused, or be an empty problem,
before anything is enqueued; struct layouts; the Python checks of shapes; memory
that a call allocates for itself."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_fp4_permute_amd as m
from tests.test_stream_memory import MAIN, SIDE, Stream, pools  # noqa: F401  (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only checks, run without a GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 20            # aligned, never dereferenced
BAD = F + 1            # misaligned
INV, UNS, WS, OK = m.ERR_INVALID, m.ERR_UNSUPPORTED, m.ERR_WORKSPACE, m.OK
I64MAX = 2 ** 63 - 1


def _route(ws=F, ws_bytes=1 << 30, **o):
    d = dict(logits=F, dtype=m.F32, T=8, E=16, k=2, score=0, renormalize=1, scale=1.0, bias=None, n_group=1, topk_group=1,
             group_top=1, topk_ids=F, topk_w=F, counts=F, offsets=F, perm_src_token=F, perm_of_assignment=F,
             perm_weight=None, scores=None)
    d.update(o)
    return m.lib().moe_route_scored(ctypes.byref(m.RouteArgs(**d)), ws, ws_bytes, None)


@pytest.mark.parametrize("o,want", [
    (dict(logits=None), INV), (dict(topk_ids=None), INV), (dict(offsets=None), INV), (dict(perm_of_assignment=None), INV),
    (dict(dtype=3), INV), (dict(T=0), INV), (dict(E=-1), INV), (dict(k=0), INV), (dict(k=17), INV), (dict(score=2), INV),
    (dict(renormalize=2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(n_group=0), INV),
    (dict(n_group=3), INV), (dict(n_group=4, topk_group=5), INV), (dict(n_group=4, topk_group=0), INV),
    (dict(n_group=4, topk_group=1, k=5), INV), (dict(group_top=0), INV), (dict(group_top=3), INV),
    (dict(n_group=16, topk_group=4, group_top=2), INV), (dict(logits=BAD), INV), (dict(dtype=m.BF16, logits=BAD), INV),
    (dict(bias=BAD), INV), (dict(scores=BAD), INV), (dict(perm_weight=BAD), INV), (dict(ws=None), WS),
    (dict(ws_bytes=16), WS), (dict(ws=F + 8), INV), (dict(E=64, k=33), UNS), (dict(E=4097), UNS),
    (dict(E=256, n_group=128, topk_group=8), UNS), (dict(T=2 ** 29), UNS), (dict(T=2 ** 25, k=1), UNS),
])
def test_route_refusals(o, want):
    assert _route(**o) == want


def _route_grad(**o):
    d = dict(logits=F, dtype=m.BF16, T=8, E=16, k=2, score=1, renormalize=0, scale=1.0, bias=None, topk_ids=F, d_topk_w=F,
             d_scores=None, d_scores_ld=0, dlogits=F)
    d.update(o)
    return m.lib().moe_route_scored_backward(ctypes.byref(m.RouteGradArgs(**d)), None)


@pytest.mark.parametrize("o,want", [
    (dict(logits=None), INV), (dict(topk_ids=None), INV), (dict(d_topk_w=None), INV), (dict(dlogits=None), INV),
    (dict(dlogits=BAD), INV), (dict(d_scores=F, d_scores_ld=8), INV), (dict(d_scores=F + 2), INV), (dict(k=20), INV),
    (dict(score=-1), INV), (dict(dtype=9), INV), (dict(E=5000), UNS), (dict(scale=float("-inf")), INV),
])
def test_route_gradient_refusals(o, want):
    assert _route_grad(**o) == want


def _combine_grad(**o):
    d = dict(dout=F, dt=m.BF16, y=F, yt=m.BF16, rows=16, perm=F, w=F, T=8, k=2, H=64, dy=F, dw=F)
    d.update(o)
    return m.lib().moe_unpermute_combine_backward(*d.values(), None)


@pytest.mark.parametrize("o,want", [
    (dict(dout=None), INV), (dict(y=None), INV), (dict(dy=None, dw=None), INV), (dict(dt=m.F16), INV), (dict(yt=5), INV),
    (dict(T=0), INV), (dict(k=0), INV), (dict(H=60), INV), (dict(rows=0), INV), (dict(rows=15, perm=None), INV),
    (dict(dout=F + 8), INV), (dict(y=F + 8), INV), (dict(dy=F + 8), INV), (dict(dw=BAD), INV), (dict(w=BAD), INV),
    (dict(perm=BAD), INV), (dict(k=1025), UNS), (dict(rows=2 ** 31), UNS), (dict(T=2 ** 24, rows=2 ** 26), UNS),
    (dict(T=2 ** 23, k=8), UNS),
])
def test_combine_gradient_refusals(o, want):
    assert _combine_grad(**o) == want


def _gemv(**o):
    d = dict(a=F, dtype=m.BF16, a_rows=None, a_rows_total=16, b_codes=F, b_scales=F, b_zeros=None, group=64, offsets=F, E=4,
             N=63, K=128, m_total=16, gated=0, activation=0, out_dtype=m.BF16, max_rows_per_expert_hint=0, out=F)
    d.update(o)
    return m.lib().int4_grouped_gemv(ctypes.byref(m.Int4GemvArgs(**d)), None)


@pytest.mark.parametrize("o,want", [
    (dict(a=None), INV), (dict(b_codes=None), INV), (dict(b_scales=None), INV), (dict(out=None), INV),
    (dict(offsets=None), INV), (dict(dtype=m.F32), INV), (dict(group=16), INV), (dict(group=0), INV), (dict(K=96), INV),
    (dict(K=0), INV), (dict(N=0), INV), (dict(N=-3), INV), (dict(E=0), INV), (dict(m_total=-1), INV),
    (dict(a_rows_total=15), INV), (dict(gated=2), INV), (dict(gated=1), INV), (dict(gated=1, N=64, activation=2), INV),
    (dict(gated=1, N=64, out_dtype=m.F32), INV), (dict(out_dtype=m.F16), INV), (dict(a=F + 8), INV), (dict(out=F + 8), INV),
    (dict(b_codes=F + 8), INV), (dict(b_scales=BAD), INV), (dict(E=4097), UNS), (dict(N=2 ** 31 - 1), UNS),
    (dict(K=2 ** 27), UNS), (dict(m_total=2 ** 30, a_rows_total=2 ** 30), UNS),
    (dict(m_total=2 ** 29, a_rows_total=2 ** 29, N=8192), UNS),
    (dict(m_total=16, max_rows_per_expert_hint=2 ** 31 - 1, N=0), INV),
    (dict(m_total=0, a=None, out=None, a_rows_total=0), OK),
])
def test_gemv_refusals(o, want):
    assert _gemv(**o) == want


def test_int4_tensor_refusals():
    q, d = m.lib().int4_quantize, m.lib().int4_dequantize
    good = [F, m.F32, 4, 64, 32, m.BF16, F, F, None, None]
    for i, v, want in ((0, None, INV), (0, F + 8, INV), (1, 4, INV), (2, 0, INV), (3, 48, INV), (3, 0, INV), (4, 48, INV),
                       (5, m.F32, INV), (6, None, INV), (6, F + 8, INV), (7, None, INV), (7, BAD, INV), (2, 2 ** 36, UNS),
                       (2, I64MAX, UNS)):
        assert q(*(good[:i] + [v] + good[i + 1:])) == want, (i, v)
    good = [F, F, None, 4, 64, 32, m.F16, m.F16, F, None]
    for i, v, want in ((0, None, INV), (1, None, INV), (3, -1, INV), (4, 40, INV), (5, 1, INV), (6, 0, INV), (7, m.BF16, INV),
                       (8, None, INV), (8, F + 8, INV), (3, 2 ** 40, UNS)):
        assert d(*(good[:i] + [v] + good[i + 1:])) == want, (i, v)


def test_null_arguments():
    L = m.lib()
    assert L.moe_route_scored(None, F, 1 << 20, None) == INV and L.moe_route_scored_backward(None, None) == INV
    assert L.int4_grouped_gemv(None, None) == INV


@pytest.mark.parametrize("cls,struct", [(m.RouteArgs, "nvfp4moe_route_args"), (m.RouteGradArgs, "nvfp4moe_route_grad_args"),
                                        (m.Int4GemvArgs, "nvfp4moe_int4_gemv_args")])
def test_structs_mirror_the_header(cls, struct):
    text = open(os.path.join(ROOT, "include", "nvfp4moe.h")).read()
    end = text.index("} " + struct + ";")
    body = re.sub(r"/\*.*?\*/", "", text[text.rindex("typedef struct", 0, end):end], flags=re.S)
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    fields = []
    for line in body.split("{", 1)[1].split(";"):
        if line.strip():
            typ, names = re.match(r"\s*((?:const\s+)?\w+\s*\*?)\s*(.+)", line.strip()).groups()
            fields += [(n.strip(), ctypes.c_void_p if "*" in typ else kinds[typ.strip()]) for n in names.split(",")]
    assert fields == list(cls._fields_)


# ------------------------------------------------------------------ the Python calls
E, H, I, T, K = 4, 64, 32, 8, 2
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _q(rows, cols, dtype=BF, group=32, zeros=False):
    lead = (E, rows)
    return m.INT4Tensor(torch.zeros(lead + (cols // 2,), dtype=U8), torch.ones(lead + (cols // group,), dtype=dtype),
                        torch.zeros(lead + (cols // group,), dtype=U8) if zeros else None, group)


def _ops():
    off = torch.tensor([0, 4, 8, 8, 16], dtype=I32)
    return dict(logits=torch.zeros((T, E)), ids=torch.zeros((T, K), dtype=I32), dw=torch.zeros((T, K)), off=off,
                x=torch.zeros((T * K, H), dtype=BF), b=_q(2 * I, H), w=torch.zeros((E, 2 * I, H)),
                dout=torch.zeros((T, H), dtype=BF), y=torch.zeros((T * K, H), dtype=BF),
                perm=torch.arange(T * K, dtype=I32))


def _fields(t):
    return tuple(v for v in vars(t).values() if isinstance(v, torch.Tensor))


CALLS = {
    "route": lambda o, s: _fields((r := m.moe_route_scored(o["logits"], K, save_scores=True, stream=s))[0]) + (r[1],),
    "route_backward": lambda o, s: (m.moe_route_scored_backward(o["dw"], o["logits"], o["ids"], stream=s),),
    "combine_backward": lambda o, s: m.moe_unpermute_combine_backward(o["dout"], o["y"], o["perm"], o["dw"], stream=s),
    "quantize": lambda o, s: _fields(m.int4_quantize(o["w"], 32, True, stream=s)),
    "dequantize": lambda o, s: (m.int4_dequantize(o["b"], stream=s),),
    "gemv": lambda o, s: (m.int4_grouped_gemv(o["x"], o["b"], o["off"], m_total=T * K, stream=s),),
    "gemv_gated": lambda o, s: (m.int4_grouped_gemv(o["x"], o["b"], o["off"], m_total=T * K, gated=True, stream=s),),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_calls_memory_comes_from_the_pool_of_its_stream(pools, name):  # noqa: F811
    o = _ops()
    pools["alloc"].clear()
    results = CALLS[name](o, Stream(SIDE))
    assert pools["calls"] == 1 and len(pools["alloc"]) >= len(results)
    assert {s for s, _ in pools["alloc"]} == {SIDE}
    for r in results:
        assert any(s == MAIN and t is r for s, t in pools["held"])


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(pools, name):  # noqa: F811
    o = _ops()
    pools["alloc"].clear()
    CALLS[name](o, None)
    assert pools["calls"] == 1 and {s for s, _ in pools["alloc"]} == {MAIN} and not pools["held"]


@pytest.fixture
def no_launch(monkeypatch):
    """The Python checks of shapes and types, on CPU tensors; a call that reaches the library fails."""
    def need(t, dtype, name, device=None):
        if t.dtype != dtype:
            raise TypeError(name)
        if not t.is_contiguous():
            raise ValueError(name)

    def reached(*a):
        raise AssertionError("not refused")
    monkeypatch.setattr(m, "_need", need)
    monkeypatch.setattr(m, "_call", reached)


REFUSED = {
    "logits_3d": lambda o: m.moe_route_scored(o["logits"][None], K),
    "logits_type": lambda o: m.moe_route_scored(o["logits"].double(), K),
    "logits_strided": lambda o: m.moe_route_scored(o["logits"].t().contiguous().t(), K),
    "bias_shape": lambda o: m.moe_route_scored(o["logits"], K, bias=torch.zeros(E + 1)),
    "bias_type": lambda o: m.moe_route_scored(o["logits"], K, bias=torch.zeros(E, dtype=BF)),
    "routing_of_another_k": lambda o: m.moe_route_scored(o["logits"], K, out=m._new_routing(T, E, K + 1, "cpu", None)),
    "routing_of_another_T": lambda o: m.moe_route_scored(o["logits"], K, out=m._new_routing(T - 1, E, K, "cpu", None)),
    "scores_shape": lambda o: m.moe_route_scored(o["logits"], K, scores=torch.zeros((T, E + 1))),
    "ids_shape": lambda o: m.moe_route_scored_backward(o["dw"], o["logits"], o["ids"][:-1].contiguous()),
    "dw_shape": lambda o: m.moe_route_scored_backward(o["dw"][:, :1].contiguous(), o["logits"], o["ids"]),
    "dw_type": lambda o: m.moe_route_scored_backward(o["dw"].to(BF), o["logits"], o["ids"]),
    "d_scores_shape": lambda o: m.moe_route_scored_backward(o["dw"], o["logits"], o["ids"], d_scores=torch.zeros((T, E + 1))),
    "d_scores_row": lambda o: m.moe_route_scored_backward(o["dw"], o["logits"], o["ids"], d_scores=torch.zeros(T + E)),
    "dlogits_type": lambda o: m.moe_route_scored_backward(o["dw"], o["logits"], o["ids"], dlogits=torch.zeros((T, E), dtype=BF)),
    "combine_h": lambda o: m.moe_unpermute_combine_backward(o["dout"][:, :32].contiguous(), o["y"], o["perm"], o["dw"]),
    "combine_w": lambda o: m.moe_unpermute_combine_backward(o["dout"], o["y"], o["perm"], o["dw"][:-1].contiguous()),
    "combine_perm": lambda o: m.moe_unpermute_combine_backward(o["dout"], o["y"], o["perm"][:-1], o["dw"]),
    "combine_rows": lambda o: m.moe_unpermute_combine_backward(o["dout"], o["y"][:-1], None, o["dw"]),
    "combine_none": lambda o: m.moe_unpermute_combine_backward(o["dout"], o["y"], o["perm"], o["dw"], need_dy=False, need_dw=False),
    "combine_f16": lambda o: m.moe_unpermute_combine_backward(o["dout"].half(), o["y"], o["perm"], o["dw"]),
    "quantize_group": lambda o: m.int4_quantize(o["w"], 48),
    "quantize_cols": lambda o: m.int4_quantize(o["w"], 128),
    "quantize_type": lambda o: m.int4_quantize(o["w"].double(), 32),
    "quantize_scales": lambda o: m.int4_quantize(o["w"], 32, scale_dtype=F32),
    "quantize_out_zeros": lambda o: m.int4_quantize(o["w"], 32, True, out=_q(2 * I, H)),
    "quantize_out_group": lambda o: m.int4_quantize(o["w"], 64, out=_q(2 * I, H)),
    "dequantize_type": lambda o: m.int4_dequantize(o["b"], torch.float16),
    "dequantize_scales": lambda o: m.int4_dequantize(m.INT4Tensor(o["b"].codes, o["b"].scales[:, :, :1].contiguous(), None, 32)),
    "gemv_type": lambda o: m.int4_grouped_gemv(o["x"].half(), o["b"], o["off"], m_total=T),
    "gemv_k": lambda o: m.int4_grouped_gemv(o["x"][:, :32].contiguous(), o["b"], o["off"], m_total=T),
    "gemv_rows": lambda o: m.int4_grouped_gemv(o["x"], o["b"], o["off"], m_total=T * K + 1),
    "gemv_offsets": lambda o: m.int4_grouped_gemv(o["x"], o["b"], o["off"][:-1], m_total=T),
    "gemv_zeros": lambda o: m.int4_grouped_gemv(o["x"], m.INT4Tensor(o["b"].codes, o["b"].scales, torch.zeros((E, 1), dtype=U8), 32),
                                                o["off"], m_total=T),
    "gemv_gated_f32": lambda o: m.int4_grouped_gemv(o["x"], o["b"], o["off"], m_total=T, gated=True, out_dtype=F32),
    "gemv_gated_odd": lambda o: m.int4_grouped_gemv(o["x"], _q(2 * I + 1, H), o["off"], m_total=T, gated=True),
    "gemv_out": lambda o: m.int4_grouped_gemv(o["x"], o["b"], o["off"], m_total=T, out=torch.zeros((T, I), dtype=BF)),
}


@pytest.mark.parametrize("name", REFUSED)
def test_python_refusals(no_launch, name):
    with pytest.raises((ValueError, TypeError)):
        REFUSED[name](_ops())
