"""The combine's gradients without weights and a layer's scores, on the host side (no GPU
needed; the library calls are left out): arguments that pass and that are refused."""
import pytest
import torch

import block_scaled_fp4_permute_amd as m

T, H, K = 6, 64, 3
BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(m, "_need", lambda t, dtype, name, device=None: None)
    monkeypatch.setattr(m, "_call", lambda dev, stream, fn, *args: seen.append(args))
    return seen


def _ops():
    return torch.zeros((T, H), dtype=BF), torch.zeros((T * K, H), dtype=BF), torch.zeros(T * K, dtype=torch.int32)


def test_no_weights(calls):
    dout, y, perm = _ops()
    for p in (perm, None):
        dy, dw = m.moe_unpermute_combine_backward(dout, y, p, None, k=K)
        assert dy.shape == y.shape and dw.shape == (T, K)
        # ..., perm, topk_w, T, k, H, dy, d_topk_w
        assert not calls[-1][6] and calls[-1][7:10] == (T, K, H) and bool(calls[-1][5]) == (p is not None)


@pytest.mark.parametrize("how", ["no_k", "perm", "rows", "another_k"])
def test_refusals(calls, how):
    dout, y, perm = _ops()
    with pytest.raises(ValueError):
        if how == "no_k":
            m.moe_unpermute_combine_backward(dout, y, perm, None)
        elif how == "perm":
            m.moe_unpermute_combine_backward(dout, y, perm, None, k=K + 1)
        elif how == "rows":
            m.moe_unpermute_combine_backward(dout, y[:-1], None, None, k=K)
        else:
            m.moe_unpermute_combine_backward(dout, y, perm, torch.zeros((T, K)), k=K - 1)
    assert not calls
