"""Memory that a call allocates for itself, on the host side (no GPU needed): it
comes from the pool of the stream that the call works on.  A block of another
stream's pool may have been freed with work still queued there that reads or
writes it, and nothing orders that work before the call's.  Results are held
for the caller's stream as well.  The library calls are replaced by a recorder;
the tensors lie on the CPU."""
import contextlib

import pytest
import torch

import block_scaled_fp4_permute_amd as m

E, H, I, T = 2, 64, 32, 16
MAIN, SIDE = "main", "side"


class Stream:
    def __init__(self, name):
        self.name, self.device, self.cuda_stream = name, torch.device("cpu"), 0

    def __eq__(self, other):
        return self.name == other.name


class _Recorder:
    """The library with its calls recorded; sizes are the real ones."""
    def __init__(self, real, launched):
        self.real, self.launched = real, launched

    def __getattr__(self, name):
        return getattr(self.real, name) if name.endswith("_size") else self.launched


@pytest.fixture
def pools(monkeypatch):
    """Allocations as (stream that was current, bytes); streams that blocks are held for; launches."""
    seen = {"alloc": [], "held": [], "calls": 0}
    current = [Stream(MAIN)]

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s or current[0]
        yield
        current[0] = before

    def recording(make):
        def f(*a, **k):
            t = make(*a, **k)
            seen["alloc"].append((current[0].name, t))
            return t
        return f

    def launched(*a):
        seen["calls"] += 1
        return m.OK

    def held(t, s):
        seen["held"].append((s.name, t))

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch, "empty", recording(torch.empty))
    monkeypatch.setattr(torch, "ones", recording(torch.ones))
    monkeypatch.setattr(torch.Tensor, "new_empty", recording(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", held)
    monkeypatch.setattr(m, "_need", lambda t, dtype, name, device=None: None)
    monkeypatch.setattr(m, "_call", launched)
    monkeypatch.setattr(m, "lib", lambda real=m.lib(): _Recorder(real, launched))
    return seen


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _operands():
    bf = torch.bfloat16
    off = torch.tensor([0, 8, T], dtype=torch.int32)
    return dict(x=torch.zeros((T, H), dtype=bf), w=torch.zeros((E, 2 * I, H), dtype=bf), off=off,
                dh=torch.zeros((T, I), dtype=bf), gu=torch.zeros((T, 2 * I)), dy=torch.zeros((T, 2 * I), dtype=bf),
                logits=torch.zeros((T, E)), g=torch.ones(E), perm=torch.zeros(T, dtype=torch.int32),
                x4=m.NVFP4Tensor(_u8(T, H // 2), _u8(T, H // 16), torch.ones(1)),
                w4=m.NVFP4Tensor(_u8(E, 2 * I, H // 2), _u8(E, 2 * I, H // 16), torch.ones(E)), packed=_u8(1 << 18),
                xm=m.MXFP4Tensor(_u8(T, H // 2), _u8(T, H // 32)), wm=m.MXFP4Tensor(_u8(E, 2 * I, H // 2), _u8(E, 2 * I, H // 32)),
                x8=torch.zeros((T, 128), dtype=bf), gu8=torch.zeros((T, 256), dtype=bf), w8=_u8(E, 256, 128),
                a8=m.FP8Tensor(_u8(T, 128), torch.ones((T, 1)), 1), s8=torch.ones((E, 2, 1)),
                q=m.INT8Tensor(torch.zeros((T, H), dtype=torch.int8), torch.ones(T)),
                wq=m.INT8Tensor(torch.zeros((E, 2 * I, H), dtype=torch.int8), torch.ones((E, 2 * I))))


def _fields(t):
    return tuple(vars(t).values())


CALLS = {
    "gated": lambda o, s: m.moe_gated_ffn(o["x"], o["w"], o["off"], m_total=T, save_gu=True, stream=s),
    "gated_backward": lambda o, s: m.moe_gated_ffn_backward(o["dh"], o["gu"], o["x"], o["w"], o["off"], stream=s),
    "product": lambda o, s: (m.moe_grouped_gemm(o["x"], o["w"], o["off"], m_total=T, stream=s),),
    "product_backward": lambda o, s: m.moe_grouped_gemm_backward(o["dy"], o["x"], o["w"], o["off"], stream=s),
    "int8_quantize": lambda o, s: (lambda q: (q.codes, q.scales))(m.int8_quantize(o["x"], stream=s)),
    "int8_product": lambda o, s: (m.int8_grouped_gemm(o["q"], o["wq"], o["off"], m_total=T, stream=s),),
    "route": lambda o, s: _fields(m.moe_route_permute(o["logits"], 2, stream=s)),
    "quantize": lambda o, s: _fields(m.nvfp4_quantize(o["x"], stream=s)),
    "route_quantize": lambda o, s: sum(map(_fields, m.moe_route_quantize(o["logits"], 2, o["x"], stream=s)), ()),
    "repack": lambda o, s: (m.nvfp4_weight_repack(o["w4"].codes, o["w4"].scales, stream=s),),
    "nvfp4": lambda o, s: (m.nvfp4_grouped_gemm(o["x4"], o["w4"].codes, o["w4"].scales, o["g"], o["off"], m_total=T,
                                                stream=s),),
    "nvfp4_swiglu": lambda o, s: _fields(m.nvfp4_grouped_gemm(
        o["x4"], o["w4"].codes, o["w4"].scales, o["g"], o["off"], m_total=T, epilogue=m.EPI_SWIGLU_NVFP4,
        out_g=o["g"], stream=s))[:2],
    "ffn": lambda o, s: (lambda r: _fields(r[0])[:2] + r[1:])(m.moe_expert_ffn(
        o["x4"], o["perm"], o["off"], o["packed"], o["g"], o["packed"], o["g"], o["g"], H=H, I=I, m_total=T,
        perm_of_assignment=o["perm"], topk_w=o["gu"], k=2, stream=s)),
    "mx_quantize": lambda o, s: _fields(m.mxfp4_quantize(o["x"], stream=s)),
    "mx_repack": lambda o, s: (m.mxfp4_weight_repack(o["wm"], stream=s),),
    "mx": lambda o, s: (m.mxfp4_grouped_gemm(o["xm"], o["wm"], o["off"], m_total=T, stream=s),),
    "mx_swiglu": lambda o, s: _fields(m.mxfp4_grouped_gemm(o["xm"], o["wm"], o["off"], m_total=T,
                                                           epilogue=m.EPI_SWIGLU_NVFP4, stream=s)),
    "fp8_quantize": lambda o, s: _fields(m.fp8_quantize(o["x8"], stream=s))[:2],
    "fp8_swiglu": lambda o, s: _fields(m.fp8_swiglu_quantize(o["gu8"], stream=s))[:2],
    "fp8_repack": lambda o, s: (m.fp8_weight_repack(o["w8"], stream=s),),
    "fp8": lambda o, s: (m.fp8_grouped_gemm(o["a8"], o["packed"], o["s8"], o["off"], N=256, m_total=T, stream=s),),
    "fp8_gated": lambda o, s: _fields(m.fp8_grouped_gemm(o["a8"], o["packed"], o["s8"], o["off"], N=256, m_total=T,
                                                         epilogue=m.EPI_SWIGLU_NVFP4, stream=s))[:2],
    "swiglu": lambda o, s: _fields(m.moe_swiglu(o["gu"], stream=s)),
    "combine": lambda o, s: (m.moe_unpermute_combine(o["dy"], None, None, T // 2, 2, stream=s),),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_calls_memory_comes_from_the_pool_of_its_stream(pools, name):
    o = _operands()
    pools["alloc"].clear()
    results = CALLS[name](o, Stream(SIDE))
    assert pools["calls"] == 1 and len(pools["alloc"]) >= len(results)
    assert {s for s, _ in pools["alloc"]} == {SIDE}
    for r in results:                       # the caller reads them on its own stream
        assert any(s == MAIN and t is r for s, t in pools["held"])


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(pools, name):
    o = _operands()
    pools["alloc"].clear()
    CALLS[name](o, None)
    assert pools["calls"] == 1 and {s for s, _ in pools["alloc"]} == {MAIN} and not pools["held"]
