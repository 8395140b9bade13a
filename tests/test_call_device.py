"""Calls on tensors of a device that is not the current one, on the host side
(no GPU needed): each call that the 16-bit and INT8 layers make runs with its
operands' device current and on that device's current stream, and a stream of
another device is refused before anything is enqueued.  The library calls and
torch's device state are replaced by recorders; the tensors lie on the CPU and
say that they are on the second GPU."""
import contextlib

import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd import layer as L

T, H, I, E, K = 8, 64, 32, 4, 2
SECOND = torch.device("cuda", 1)


class OnSecond(torch.Tensor):
    """A CPU tensor that claims to be on the second GPU."""
    device = property(lambda self: SECOND)
    is_cuda = property(lambda self: True)


def _second(make):
    def f(*a, **k):
        k.pop("device", None)
        return make(*a, **k).as_subclass(OnSecond)
    return f


class _Stream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 1000 + index


@pytest.fixture
def launches(monkeypatch):
    """(library call, current device, raw stream) of every launch; the first GPU is current."""
    current, seen, real = [0], [], m.lib()

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real, name)
            return lambda *a: seen.append((name, current[0], a[-1])) or m.OK

    monkeypatch.setattr(m, "lib", lambda: Lib())
    monkeypatch.setattr(torch, "empty", _second(torch.empty))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: _Stream(current[0] if d is None else d.index))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    return seen


def _weights():
    bf = torch.bfloat16
    return (torch.empty((T, E), dtype=torch.float32), torch.empty((T, H), dtype=bf), torch.empty((E, 2 * I, H), dtype=bf),
            torch.empty((E, H, I), dtype=bf))


def test_layer16_on_a_device_that_is_not_current(launches):
    logits, x, w_gu, w_dn = _weights()
    layer = L.MoELayer16(T, H, I, E, K, SECOND)
    layer.forward(logits, x, w_gu, w_dn)
    gu = torch.empty((T * K, 2 * I), dtype=torch.float32)
    layer.expert_rows(x, w_gu, w_dn, gu=gu)
    layer.expert_rows_backward(layer.y2, gu, x, w_gu, w_dn)
    assert [n for n, _, _ in launches] == ["moe_route_permute", "moe_gated_ffn", "moe_grouped_gemm", "moe_unpermute_combine",
                                           "moe_gated_ffn", "moe_grouped_gemm", "moe_grouped_gemm_backward",
                                           "moe_gated_ffn_backward", "moe_unpermute_combine"]
    assert all(d == 1 and s == 1001 for _, d, s in launches), launches


def test_int8_layer_on_a_device_that_is_not_current(launches):
    logits, x, w_gu, w_dn = _weights()
    w = L.quantize_expert_weights_int8(w_gu, w_dn)
    L.INT8MoELayer(T, H, I, E, K, SECOND).forward(logits, x, w)
    assert len(launches) == 8 and all(d == 1 and s == 1001 for _, d, s in launches), launches


def test_a_stream_of_another_device_is_refused(launches):
    logits, x, w_gu, w_dn = _weights()
    off = torch.empty(E + 1, dtype=torch.int32)
    for call in (lambda s: m.moe_gated_ffn(x, w_gu, off, m_total=T, stream=s),
                 lambda s: m.moe_grouped_gemm(x, w_gu, off, m_total=T, stream=s),
                 lambda s: m.int8_quantize(x, stream=s), lambda s: m.moe_route_permute(logits, K, stream=s),
                 lambda s: m.moe_unpermute_combine(x, None, None, T // K, K, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(_Stream(0))
        assert not launches
        call(_Stream(1))
        assert [(d, s) for _, d, s in launches] == [(1, 1001)]
        launches.clear()
