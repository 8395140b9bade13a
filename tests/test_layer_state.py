"""MoELayer16 keeps h and the routing of its last call for expert_rows_backward,
on the host side (no GPU needed; the library calls are left out): gradients of
a call whose h or routing is no longer there are refused."""
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from block_scaled_fp4_permute_amd.layer import MoELayer16

T, H, I, E, K = 8, 64, 32, 4, 2
BF = torch.bfloat16


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(m, "_need", lambda t, dtype, name, device=None: None)
    monkeypatch.setattr(m, "_call", lambda *a: None)
    return MoELayer16(T, H, I, E, K, "cpu")


def _operands():
    return (torch.zeros((T, H), dtype=BF), torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, H, I), dtype=BF))


def _gu():
    return torch.zeros((T * K, 2 * I))


def test_gradients_of_the_last_call(layer):
    ops, gu, dy = _operands(), _gu(), torch.zeros((T * K, H), dtype=BF)
    layer.route(torch.zeros((T, E)))
    layer.expert_rows(*ops, gu=gu)
    for _ in range(2):
        assert len(layer.expert_rows_backward(dy, gu, *ops)) == 3
    layer.expert_rows(*ops, gu=gu)
    assert len(layer.expert_rows_backward(dy, gu, *ops)) == 3


@pytest.mark.parametrize("between", ["nothing", "another_batch", "no_gu", "forward", "route", "failed_call"])
def test_gradients_of_another_call_are_refused(layer, between):
    ops, gu, dy, logits = _operands(), _gu(), torch.zeros((T * K, H), dtype=BF), torch.zeros((T, E))
    if between != "nothing":
        layer.route(logits)
        layer.expert_rows(*ops, gu=gu)
    other = _gu()
    if between == "another_batch":
        layer.expert_rows(*ops, gu=other)
    elif between == "no_gu":
        layer.expert_rows(*ops)
    elif between == "forward":
        layer.forward(logits, *ops)
    elif between == "route":
        layer.route(logits)
    elif between == "failed_call":
        with pytest.raises(ValueError):
            layer.expert_rows(ops[0], ops[1], ops[2][:, :, :8].contiguous(), gu=gu)
    with pytest.raises(ValueError, match="expert_rows"):
        layer.expert_rows_backward(dy, gu, *ops)
    if between == "another_batch":
        assert len(layer.expert_rows_backward(dy, other, *ops)) == 3


def test_float16_forward_is_refused_before_anything_runs(monkeypatch):
    """The combine takes no float16 rows; expert_rows is for those."""
    ran = []
    monkeypatch.setattr(m, "_need", lambda t, dtype, name, device=None: None)
    monkeypatch.setattr(m, "_call", lambda *a: ran.append(a))
    layer = MoELayer16(T, H, I, E, K, "cpu", dtype=torch.float16)
    x, w_gu, w_dn = (t.half() for t in _operands())
    with pytest.raises(TypeError, match="float16"):
        layer.forward(torch.zeros((T, E)), x, w_gu, w_dn)
    assert not ran
    layer.route(torch.zeros((T, E)))
    assert layer.expert_rows(x, w_gu, w_dn).dtype == torch.float16
