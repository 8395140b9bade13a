"""Host-side checks of the 16-bit expert FFN, INT8 and their gradients (no GPU
needed): every call below has to be refused, or be an empty problem, before
anything is enqueued.  Struct layouts are checked against the header's."""
import ctypes
import os
import re

import pytest

import block_scaled_fp4_permute_amd as m

try:
    import torch
    _HAVE_GPU = torch.cuda.is_available()
except Exception:  # pragma: no cover
    _HAVE_GPU = False
pytestmark = pytest.mark.skipif(_HAVE_GPU, reason="fake device addresses: host-only checks, run without a GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 20            # aligned, never dereferenced
BAD = F + 4            # misaligned
I32MAX, I64MAX = 2 ** 31 - 1, 2 ** 63 - 1
INV, UNS, WS, OK = m.ERR_INVALID, m.ERR_UNSUPPORTED, m.ERR_WORKSPACE, m.OK


def _gated(**o):
    d = dict(x=F, dtype=m.BF16, a_rows=None, x_rows=16, w=F, offsets=F, E=4, H=64, I=32, m_total=16, activation=0,
             max_rows_per_expert_hint=0, h=F, gu=None)
    d.update(o)
    return m.lib().moe_gated_ffn(ctypes.byref(m.GatedArgs(**d)), None)


def _gated_grad(ws=F, ws_bytes=None, **o):
    d = dict(x=F, dtype=m.BF16, a_rows=None, x_rows=16, w=F, offsets=F, E=4, H=64, I=32, m_total=16, activation=0,
             max_rows_per_expert_hint=0, gu=F, dh=F, dx=F, dw=F)
    d.update(o)
    if ws_bytes is None:
        ws_bytes = m.lib().moe_gated_ffn_backward_workspace_size(4, 64, 32, 16)
    return m.lib().moe_gated_ffn_backward(ctypes.byref(m.GatedGradArgs(**d)), ws, ws_bytes, None)


def _product(**o):
    d = dict(a=F, dtype=m.F16, a_rows=None, a_rows_total=16, b=F, offsets=F, E=4, N=64, K=32, m_total=16,
             out_dtype=m.F16, max_rows_per_expert_hint=0, out=F)
    d.update(o)
    return m.lib().moe_grouped_gemm(ctypes.byref(m.ProductArgs(**d)), None)


def _product_grad(**o):
    d = dict(a=F, dtype=m.F16, a_rows=None, a_rows_total=16, b=F, offsets=F, E=4, N=64, K=32, m_total=16,
             max_rows_per_expert_hint=0, dy=F, da=F, db=F)
    d.update(o)
    return m.lib().moe_grouped_gemm_backward(ctypes.byref(m.ProductGradArgs(**d)), None, 0, None)


def _int8(**o):
    d = dict(a_codes=F, a_scales=F, a_rows=None, a_rows_total=16, b_codes=F, b_scales=F, offsets=F, E=4, N=64, K=32,
             m_total=16, epilogue=m.EPI_BF16, max_rows_per_expert_hint=0, out=F)
    d.update(o)
    return m.lib().int8_grouped_gemm(ctypes.byref(m.Int8GemmArgs(**d)), None)


@pytest.mark.parametrize("o,want", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(h=None), INV), (dict(offsets=None), INV), (dict(dtype=m.F32), INV),
    (dict(E=0), INV), (dict(H=0), INV), (dict(I=0), INV), (dict(H=60), INV), (dict(I=36), INV), (dict(I=-8), INV),
    (dict(m_total=-1), INV), (dict(x_rows=-1), INV), (dict(x_rows=15), INV), (dict(x_rows=0, a_rows=F), INV),
    (dict(activation=2), INV), (dict(x=BAD), INV), (dict(w=BAD), INV), (dict(h=BAD), INV), (dict(gu=BAD), INV),
    (dict(a_rows=F + 2), INV), (dict(E=5000), UNS), (dict(m_total=2 ** 31, x_rows=2 ** 31), UNS),
    (dict(I=2 ** 26), UNS), (dict(H=2 ** 27), UNS), (dict(I=I32MAX - 7, H=I32MAX - 7), UNS),
    (dict(m_total=I64MAX, x_rows=I64MAX), UNS), (dict(m_total=2 ** 29, x_rows=2 ** 29, I=2 ** 20), UNS), (dict(m_total=2 ** 30, x_rows=2 ** 30), UNS),
    (dict(m_total=0, x=None, h=None, x_rows=0), OK),
])
def test_gated_refusals(o, want):
    assert _gated(**o) == want


@pytest.mark.parametrize("o,want", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(gu=None), INV), (dict(dh=None), INV), (dict(dx=None, dw=None), INV),
    (dict(dtype=7), INV), (dict(I=12), INV), (dict(dx=BAD), INV), (dict(dw=BAD), INV), (dict(gu=BAD), INV),
    (dict(activation=-1), INV), (dict(x_rows=3), INV), (dict(E=4097), UNS), (dict(ws=None), WS),
    (dict(ws_bytes=16 * 64 * 2), WS), (dict(ws=F + 16), INV), (dict(m_total=2 ** 31), UNS),
    (dict(m_total=0, x=None, gu=None, dh=None, dx=None, dw=None, x_rows=0, ws_bytes=1 << 20), OK),
])
def test_gated_gradient_refusals(o, want):
    assert _gated_grad(**o) == want


@pytest.mark.parametrize("o,want", [
    (dict(a=None), INV), (dict(b=None), INV), (dict(out=None), INV), (dict(out_dtype=m.BF16), INV), (dict(N=4), INV),
    (dict(K=12), INV), (dict(out=BAD), INV), (dict(a_rows_total=2), INV), (dict(dtype=m.F32, out_dtype=m.F32), INV),
    (dict(N=I32MAX - 7, K=I32MAX - 7, m_total=2 ** 30, a_rows_total=2 ** 30), UNS),
    (dict(m_total=0, a=None, out=None, a_rows_total=0), OK),
])
def test_product_refusals(o, want):
    assert _product(**o) == want


@pytest.mark.parametrize("o,want", [
    (dict(a=None), INV), (dict(b=None), INV), (dict(dy=None), INV), (dict(da=None, db=None), INV), (dict(da=BAD), INV),
    (dict(db=BAD), INV), (dict(dy=BAD), INV), (dict(a_rows_total=2), INV), (dict(E=4096, N=2 ** 20, K=2 ** 20), UNS),
    (dict(m_total=0, dy=None, a=None, da=None, db=None, a_rows_total=0), OK),
])
def test_product_gradient_refusals(o, want):
    assert _product_grad(**o) == want


@pytest.mark.parametrize("o,want", [
    (dict(a_codes=None), INV), (dict(a_scales=None), INV), (dict(b_codes=None), INV), (dict(b_scales=None), INV),
    (dict(out=None), INV), (dict(K=24), INV), (dict(K=131072), UNS), (dict(N=12), INV),
    (dict(N=24, epilogue=m.EPI_SWIGLU_BF16), INV), (dict(epilogue=m.EPI_COMBINE_F32), UNS), (dict(epilogue=9), UNS),
    (dict(a_codes=F + 8), INV), (dict(b_scales=F + 8), INV), (dict(a_scales=F + 2), INV), (dict(E=-1), INV),
    (dict(m_total=0, a_codes=None, a_scales=None, out=None, a_rows_total=0), OK),
])
def test_int8_product_refusals(o, want):
    assert _int8(**o) == want


def test_int8_quantizer_refusals():
    q = m.lib().int8_quantize
    assert q(None, m.BF16, 4, 64, F, F, None) == INV
    assert q(F, m.F16, 4, 64, F, F, None) == INV
    assert q(F, m.F32, 0, 64, F, F, None) == INV
    assert q(F, m.F32, 4, 60, F, F, None) == INV
    assert q(F + 8, m.F32, 4, 64, F, F, None) == INV
    assert q(F, m.F32, 4, 64, F + 4, F, None) == INV
    assert q(F, m.F32, 4, 64, F, F + 2, None) == INV
    assert q(F, m.F32, 2 ** 31, 64, F, F, None) == UNS
    assert q(F, m.F32, I64MAX, I64MAX - 7, F, F, None) == UNS


def test_null_arguments_and_workspace_sizes():
    L = m.lib()
    assert L.moe_gated_ffn(None, None) == INV and L.moe_grouped_gemm(None, None) == INV
    assert L.moe_gated_ffn_backward(None, F, 1 << 20, None) == INV
    assert L.moe_grouped_gemm_backward(None, None, 0, None) == INV and L.int8_grouped_gemm(None, None) == INV
    size = L.moe_gated_ffn_backward_workspace_size
    assert size(4, 64, 32, 16) >= 2 * 16 * 64 * 2 and size(4, 64, 32, 0) > 0
    for bad in ((0, 64, 32, 16), (4, 60, 32, 16), (4, 64, 12, 16), (5000, 64, 32, 16), (4, 64, 32, -1),
                (4, 64, I32MAX - 7, I64MAX)):
        assert size(*bad) == 0


@pytest.mark.parametrize("cls,struct", [
    (m.GatedArgs, "nvfp4moe_gated_args"), (m.GatedGradArgs, "nvfp4moe_gated_grad_args"),
    (m.ProductArgs, "nvfp4moe_product_args"), (m.ProductGradArgs, "nvfp4moe_product_grad_args"),
    (m.Int8GemmArgs, "nvfp4moe_int8_gemm_args")])
def test_structs_mirror_the_header(cls, struct):
    text = open(os.path.join(ROOT, "include", "nvfp4moe.h")).read()
    end = text.index("} " + struct + ";")
    body = re.sub(r"/\*.*?\*/", "", text[text.rindex("typedef struct", 0, end):end], flags=re.S)
    fields = []
    for line in body.split("{", 1)[1].split(";"):
        line = line.strip()
        if not line:
            continue
        typ, names = re.match(r"((?:const\s+)?\w+\s*\*?)\s*(.+)", line).groups()
        for n in names.split(","):
            kind = ctypes.c_void_p if "*" in typ else {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64}[typ.strip()]
            fields.append((n.strip(), kind))
    assert fields == list(cls._fields_)
